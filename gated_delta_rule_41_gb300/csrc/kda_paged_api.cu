// C ABI of the paged key-value cache and its page bookkeeping: argument
// validation.  As in kda_api.cu, a rejected call enqueues nothing.
#include <climits>
#include <cmath>

#include "kda_common.cuh"

namespace {

using namespace kda;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kMaxPages = 1 << 30;   // page ids and their scans are 32-bit

int page_shift(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Sizes and pool strides; `attend` also checks what only the attention reads.
kda_status check_dims(const kda_paged_dims* d, bool attend) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->cache_dtype != KDA_F32 && d->cache_dtype != KDA_BF16 && d->cache_dtype != KDA_E4M3)
        return KDA_ERR_INVALID_ARG;
    if (d->S < 0 || d->HKV <= 0 || d->D <= 0 || d->num_pages <= 0 || d->page_size <= 0 ||
        d->max_pages <= 0)
        return KDA_ERR_SHAPE;
    if (d->cache_dtype == KDA_F32) return KDA_ERR_UNSUPPORTED;
    if ((d->D != 64 && d->D != 128) || page_shift(d->page_size) < 0) return KDA_ERR_UNSUPPORTED;
    if (d->S > 65535 || d->HKV > 65535 || d->num_pages > kMaxPages) return KDA_ERR_UNSUPPORTED;
    if ((long long)d->max_pages * d->page_size > INT_MAX / 2) return KDA_ERR_UNSUPPORTED;
    const long long per16 = d->cache_dtype == KDA_E4M3 ? 16 : 8;
    if (d->page_stride % per16 || d->token_stride % per16 || d->head_stride % per16)
        return KDA_ERR_ALIGNMENT;
    // rows do not overlap; the stride of a dimension of one is not used
    if (d->token_stride < d->D || (d->HKV > 1 && d->head_stride < d->D) ||
        (d->num_pages > 1 && d->page_stride < d->D) || d->page_stride < 0 || d->head_stride < 0)
        return KDA_ERR_SHAPE;
    if (!attend) return KDA_OK;
    if (d->HQ <= 0 || d->HQ % d->HKV != 0) return KDA_ERR_SHAPE;
    if (d->HQ / d->HKV > 64) return KDA_ERR_UNSUPPORTED;
    if (d->window < 0 || d->sinks < 0 || !std::isfinite(d->scale)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

PagedArgs make_args(const kda_paged_dims& d) {
    PagedArgs a = {};
    a.S = d.S;
    a.HQ = d.HQ;
    a.HKV = d.HKV;
    a.G = d.HQ > 0 ? d.HQ / d.HKV : 0;
    a.num_pages = d.num_pages;
    a.page_shift = page_shift(d.page_size);
    a.max_pages = d.max_pages;
    a.cap = d.max_pages * d.page_size;
    a.page_stride = d.page_stride;
    a.token_stride = d.token_stride;
    a.head_stride = d.head_stride;
    a.scale = d.scale;
    // a window as wide as the table hides nothing (and the kernels' sums of positions and
    // windows stay in range)
    a.window = d.window < a.cap ? d.window : 0;
    a.sinks = a.window ? d.sinks : 0;
    return a;
}

// Pools, scales and tables.
kda_status check_cache(const void* kp, const void* vp, const float* ks, const float* vs,
                       const int* table, const int* lens) {
    if (!kp || !vp || !table || !lens) return KDA_ERR_INVALID_ARG;
    if (!aligned(kp, 16) || !aligned(vp, 16)) return KDA_ERR_ALIGNMENT;
    if (!aligned(ks, 4) || !aligned(vs, 4) || !aligned(table, 4) || !aligned(lens, 4))
        return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

// A token tensor [T][heads][D] bf16 whose tokens are `stride` elements apart.
kda_status check_tokens(const void* p, long long stride, int T, long long row) {
    if (!p) return KDA_ERR_INVALID_ARG;
    if (!aligned(p, 16)) return KDA_ERR_ALIGNMENT;
    if (T > 1 && stride < row) return KDA_ERR_SHAPE;
    return stride % 8 ? KDA_ERR_ALIGNMENT : KDA_OK;
}

kda_status check_attend(const kda_paged_dims* d, const int* cu, bool need_cu, int T, const void* q,
                        long long q_stride, const void* kp, const void* vp, const float* ks,
                        const float* vs, const int* table, const int* lens, const void* o,
                        const float* lse) {
    kda_status st = check_dims(d, true);
    if (st != KDA_OK) return st;
    if (T < 0) return KDA_ERR_SHAPE;
    if ((long long)T * d->HQ > INT_MAX / 2) return KDA_ERR_UNSUPPORTED;
    if (T == 0 || d->S == 0) return T == 0 ? KDA_OK : KDA_ERR_SHAPE;
    if (need_cu && !cu) return KDA_ERR_INVALID_ARG;
    if (!aligned(cu, 4) || !aligned(lse, 4)) return KDA_ERR_ALIGNMENT;
    if ((st = check_cache(kp, vp, ks, vs, table, lens)) != KDA_OK) return st;
    if ((st = check_tokens(q, q_stride, T, (long long)d->HQ * d->D)) != KDA_OK) return st;
    if (!o) return KDA_ERR_INVALID_ARG;
    return aligned(o, 16) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

kda_status check_ws(size_t need, const void* ws, size_t bytes) {
    if (need == 0) return KDA_OK;
    if (!ws || bytes < need) return KDA_ERR_WORKSPACE;
    return aligned(ws, 256) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

void fill(PagedArgs& a, const int* cu, int T, const void* q, long long q_stride, const void* kp,
          const void* vp, const float* ks, const float* vs, const int* table, const int* lens,
          void* o, float* lse) {
    a.cu = cu;
    a.T = T;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_stride = q_stride;
    a.kp = kp;
    a.vp = vp;
    a.ks = ks;
    a.vs = vs;
    a.table = table;
    a.lens = lens;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
}

kda_status check_pages_dims(const kda_pages_dims* d) {
    if (!d) return KDA_ERR_INVALID_ARG;
    if (d->S < 0 || d->max_pages <= 0 || d->num_pages <= 0 || d->page_size <= 0)
        return KDA_ERR_SHAPE;
    if (d->S > 65535 || d->num_pages > kMaxPages ||
        (long long)d->max_pages * d->page_size > INT_MAX / 2)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_pools(const kda_page_pool* pools, int n) {
    if (n < 0) return KDA_ERR_SHAPE;
    if (n > KDA_MAX_POOLS) return KDA_ERR_UNSUPPORTED;
    if (n > 0 && !pools) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (!pools[i].base) return KDA_ERR_INVALID_ARG;
        if (pools[i].page_bytes <= 0 || pools[i].page_stride_bytes < pools[i].page_bytes)
            return KDA_ERR_SHAPE;
        if (!aligned(pools[i].base, 16) || pools[i].page_bytes % 16 ||
            pools[i].page_stride_bytes % 16)
            return KDA_ERR_ALIGNMENT;
    }
    return KDA_OK;
}

kda_status check_ints(std::initializer_list<const int*> required) {
    for (const int* p : required) {
        if (!p) return KDA_ERR_INVALID_ARG;
        if (!aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_paged_append(const kda_paged_dims* d, const int* cu, int T, const void* k,
                            long long k_stride, const void* v, long long v_stride,
                            const float* ks, const float* vs, const int* table, const int* lens,
                            void* kp, void* vp, void* stream) {
    return kda_paged_append_granted(d, cu, T, k, k_stride, v, v_stride, ks, vs, table, lens,
                                    nullptr, kp, vp, stream);
}

kda_status kda_paged_append_granted(const kda_paged_dims* d, const int* cu, int T, const void* k,
                                    long long k_stride, const void* v, long long v_stride,
                                    const float* ks, const float* vs, const int* table,
                                    const int* lens, const int* granted, void* kp, void* vp,
                                    void* stream) {
    kda_status st = check_dims(d, false);
    if (st != KDA_OK) return st;
    if (T < 0 || (!cu && T != d->S)) return KDA_ERR_SHAPE;
    if ((long long)T * d->HKV > INT_MAX / 32) return KDA_ERR_UNSUPPORTED;
    if (T == 0) return KDA_OK;
    if (d->S == 0) return KDA_ERR_SHAPE;
    if (!aligned(cu, 4) || !aligned(granted, 4)) return KDA_ERR_ALIGNMENT;
    if ((st = check_cache(kp, vp, ks, vs, table, lens)) != KDA_OK) return st;
    const long long row = (long long)d->HKV * d->D;
    if ((st = check_tokens(k, k_stride, T, row)) != KDA_OK) return st;
    if ((st = check_tokens(v, v_stride, T, row)) != KDA_OK) return st;
    PagedArgs a = make_args(*d);
    fill(a, cu, T, nullptr, 0, kp, vp, ks, vs, table, lens, nullptr, nullptr);
    return paged_append_launch(a, d->D, d->cache_dtype == KDA_E4M3, k, k_stride, v, v_stride,
                               granted, static_cast<cudaStream_t>(stream));
}

size_t kda_paged_decode_workspace_bytes(const kda_paged_dims* d) {
    if (check_dims(d, true) != KDA_OK || d->S == 0) return 0;
    return paged_decode_ws_bytes(make_args(*d), d->D, d->cache_dtype == KDA_E4M3);
}

kda_status kda_paged_decode(const kda_paged_dims* d, const void* q, long long q_stride,
                            const void* kp, const void* vp, const float* ks, const float* vs,
                            const int* table, const int* lens, void* o, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
    kda_status st = check_attend(d, nullptr, false, d ? d->S : 0, q, q_stride, kp, vp, ks, vs,
                                 table, lens, o, lse);
    if (st != KDA_OK || d->S == 0) return st;
    PagedArgs a = make_args(*d);
    const bool e4m3 = d->cache_dtype == KDA_E4M3;
    if ((st = check_ws(paged_decode_ws_bytes(a, d->D, e4m3), ws, ws_bytes)) != KDA_OK) return st;
    fill(a, nullptr, d->S, q, q_stride, kp, vp, ks, vs, table, lens, o, lse);
    return paged_decode_launch(a, d->D, e4m3, ws, static_cast<cudaStream_t>(stream));
}

size_t kda_paged_prefill_workspace_bytes(const kda_paged_dims* d, int T) {
    if (check_dims(d, true) != KDA_OK || d->S == 0 || T <= 0 ||
        (long long)T * d->HQ > INT_MAX / 2)
        return 0;
    PagedArgs a = make_args(*d);
    a.T = T;
    return paged_prefill_ws_bytes(a, d->D, d->cache_dtype == KDA_E4M3);
}

kda_status kda_paged_prefill(const kda_paged_dims* d, const int* cu, int T, const void* q,
                             long long q_stride, const void* kp, const void* vp, const float* ks,
                             const float* vs, const int* table, const int* lens, void* o,
                             float* lse, void* ws, size_t ws_bytes, void* stream) {
    kda_status st = check_attend(d, cu, true, T, q, q_stride, kp, vp, ks, vs, table, lens, o, lse);
    if (st != KDA_OK || T == 0) return st;
    PagedArgs a = make_args(*d);
    fill(a, cu, T, q, q_stride, kp, vp, ks, vs, table, lens, o, lse);
    const bool e4m3 = d->cache_dtype == KDA_E4M3;
    if ((st = check_ws(paged_prefill_ws_bytes(a, d->D, e4m3), ws, ws_bytes)) != KDA_OK) return st;
    return paged_prefill_launch(a, d->D, e4m3, ws, static_cast<cudaStream_t>(stream));
}

size_t kda_pages_workspace_bytes(const kda_pages_dims* d) {
    return check_pages_dims(d) == KDA_OK ? pages_ws_bytes(*d) : 0;
}

kda_status kda_pages_fork(const kda_pages_dims* d, const kda_page_pool* pools, int num_pools,
                          const int* parents, const int* children, int n, int* table, int* lens,
                          int* refs, void* ws, size_t ws_bytes, void* stream) {
    kda_status st = check_pages_dims(d);
    if (st != KDA_OK) return st;
    if (n < 0 || n > d->S) return KDA_ERR_SHAPE;
    if ((st = check_pools(pools, num_pools)) != KDA_OK || n == 0) return st;
    if ((st = check_ints({parents, children, table, lens, refs})) != KDA_OK) return st;
    if ((st = check_ws(pages_ws_bytes(*d), ws, ws_bytes)) != KDA_OK) return st;
    return pages_fork_launch(*d, pools, num_pools, parents, children, n, table, lens, refs, ws,
                             static_cast<cudaStream_t>(stream));
}

kda_status kda_pages_extend(const kda_pages_dims* d, const int* add, int add_all, int* table,
                            int* lens, int* refs, void* ws, size_t ws_bytes, void* stream) {
    return kda_pages_extend_granted(d, add, add_all, table, lens, refs, nullptr, ws, ws_bytes,
                                    stream);
}

kda_status kda_pages_extend_granted(const kda_pages_dims* d, const int* add, int add_all,
                                    int* table, int* lens, int* refs, int* granted, void* ws,
                                    size_t ws_bytes, void* stream) {
    kda_status st = check_pages_dims(d);
    if (st != KDA_OK) return st;
    if (!add && add_all < 0) return KDA_ERR_SHAPE;
    if (d->S == 0) return KDA_OK;
    if (!aligned(add, 4) || !aligned(granted, 4)) return KDA_ERR_ALIGNMENT;
    if ((st = check_ints({table, lens, refs})) != KDA_OK) return st;
    if ((st = check_ws(pages_ws_bytes(*d), ws, ws_bytes)) != KDA_OK) return st;
    return pages_extend_launch(*d, add, add_all, table, lens, refs, granted, ws,
                               static_cast<cudaStream_t>(stream));
}

kda_status kda_pages_free(const kda_pages_dims* d, const int* slots, int n, int* table, int* lens,
                          int* refs, void* stream) {
    kda_status st = check_pages_dims(d);
    if (st != KDA_OK) return st;
    if (n < 0 || n > d->S) return KDA_ERR_SHAPE;
    if (n == 0) return KDA_OK;
    if ((st = check_ints({slots, table, lens, refs})) != KDA_OK) return st;
    return pages_free_launch(*d, slots, n, table, lens, refs, static_cast<cudaStream_t>(stream));
}

kda_status kda_pages_compact(const kda_pages_dims* d, const kda_page_pool* pools, int num_pools,
                             int* table, int* refs, void* ws, size_t ws_bytes, void* stream) {
    kda_status st = check_pages_dims(d);
    if (st != KDA_OK) return st;
    if ((st = check_pools(pools, num_pools)) != KDA_OK) return st;
    if ((st = check_ints({refs})) != KDA_OK) return st;
    if (d->S > 0 && (st = check_ints({table})) != KDA_OK) return st;
    if ((st = check_ws(pages_ws_bytes(*d), ws, ws_bytes)) != KDA_OK) return st;
    return pages_compact_launch(*d, pools, num_pools, table, refs, ws,
                                static_cast<cudaStream_t>(stream));
}

kda_status kda_pages_copy(const kda_page_pool* pools, int num_pools, int num_pages,
                          const int* src, const int* dst, int n, void* stream) {
    if (n < 0 || num_pages <= 0) return KDA_ERR_SHAPE;
    kda_status st = check_pools(pools, num_pools);
    if (st != KDA_OK || n == 0 || num_pools == 0) return st;
    if ((st = check_ints({src, dst})) != KDA_OK) return st;
    return pages_copy_launch(pools, num_pools, num_pages, src, dst, n,
                             static_cast<cudaStream_t>(stream));
}

}  // extern "C"
