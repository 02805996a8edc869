// Paged key-value cache: appending tokens.
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_paged.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_paged_error = 0;   // a kda_status

namespace {

__device__ __forceinline__ void record() { atomicCAS(&g_paged_error, 0, (int)KDA_ERR_SHAPE); }

__device__ __forceinline__ int seq_len(const PagedArgs& a, int s) {
    const int len = a.lens[s];
    if (len < 0 || len > a.cap) {
        record();
        return 0;
    }
    return len;
}

// Eight e4m3 codes of x * inv, saturated at +-448.
__device__ __forceinline__ uint2 quant8(const uint4 v, float inv) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    uint2 r;
    unsigned short* c = reinterpret_cast<unsigned short*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f = __bfloat1622float2(h[i]);
        f.x *= inv;
        f.y *= inv;
        c[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return r;
}

// A pass of copies bounded by HBM: T (HKV D) (2 + code) bytes each of K and V.
// A CTA takes TB tokens, whole rows of K and V, as items that end in one 16-byte
// store: eight elements, or sixteen from two loads for e4m3 (41 us below with
// eight).  Its first items are on their way before the tokens' places are looked up
// (sequence, length, table entry: three dependent reads), so that the copies do
// not wait for them.  32k tokens of 8 heads of 128 into e4m3 pages, 194 MB: 35 us,
// 5.5 TB/s (one warp per row and head, each with its own look-up: 66 us); 256
// single tokens 2.4 us.
constexpr int kAppendThreads = 256, kAppendItems = 8;   // of a thread at a time
constexpr int kAppendTokens = 64;                       // of a CTA, at most
constexpr int kAppendHeads = 128;                       // whose inverse scales are kept

template <int D, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const PagedArgs a, int TB, const __nv_bfloat16* __restrict__ k, long long k_stride,
              const __nv_bfloat16* __restrict__ v, long long v_stride, const int* granted) {
    __shared__ int s_seq[kAppendTokens];
    __shared__ long long s_off[kAppendTokens];          // element of the token's row, or -1
    __shared__ float s_inv[2 * kAppendHeads];           // 1 / scale of K, V per head
    const int tid = threadIdx.x, t0 = blockIdx.x * TB, n = min(TB, a.T - t0);
    constexpr int V = E4M3 ? 2 : 1, EL = 8 * V;         // 16-byte loads, elements of an item
    const int row = a.HKV * (D / EL), per = 2 * row;    // items of a row of K, of a token

    // A thread's items lie kAppendThreads apart: (token, item of it), stepped
    // without a division.
    const int step_tok = kAppendThreads / per, step_at = kAppendThreads % per;
    auto step = [&](int& tok, int& at) {
        tok += step_tok;
        at += step_at;
        if (at >= per) {
            at -= per;
            ++tok;
        }
    };
    constexpr int kItems = kAppendItems / V;
    uint4 x[kItems][V];
    int tok0 = tid / per, at0 = tid % per;              // of the thread's first item of a round
    auto load = [&]() {
        int tok = tok0, at = at0;
#pragma unroll
        for (int i = 0; i < kItems; ++i, step(tok, at)) {
            if (tok >= n) continue;
            const long long t = t0 + tok;
            const uint4* src = reinterpret_cast<const uint4*>(
                at < row ? k + t * k_stride + (long long)EL * at
                         : v + t * v_stride + (long long)EL * (at - row));
#pragma unroll
            for (int e = 0; e < V; ++e) x[i][e] = __ldcs(src + e);
        }
    };
    load();

    if (E4M3) {
        for (int i = tid; i < 2 * min(a.HKV, kAppendHeads); i += kAppendThreads) {
            const float* sc = i & 1 ? a.vs : a.ks;
            s_inv[i] = sc ? 1.0f / sc[i >> 1] : 1.0f;
        }
    }
    if (a.cu) {
        // who owns the tokens; cu must rise from 0 to T
        bool bad = tid == 0 && (a.cu[0] != 0 || a.cu[a.S] != a.T);
        for (int i = tid; i < a.S; i += kAppendThreads) {
            const int lo = a.cu[i], hi = a.cu[i + 1];
            bad |= lo < 0 || lo > hi || hi > a.T;
            if (bad) break;
            for (int t = max(lo, t0); t < min(hi, t0 + n); ++t) s_seq[t - t0] = i;
        }
        if (__syncthreads_or(bad)) {
            if (tid == 0) record();
            return;
        }
    }
    if (tid < n) {
        const int t = t0 + tid, s = a.cu ? s_seq[tid] : t;
        const int pos = seq_len(a, s) - (a.cu ? a.cu[s + 1] - t : 1);
        // before the sequence's start, or meant for a refused row: dropped
        long long off = -1;
        if (pos >= 0 && (!granted || granted[s] > 0)) {
            const int page = a.table[(size_t)s * a.max_pages + (pos >> a.page_shift)];
            if ((unsigned)page < (unsigned)a.num_pages)
                off = page * a.page_stride + (pos & ((1 << a.page_shift) - 1)) * a.token_stride;
            else
                record();
        }
        s_off[tid] = off;
    }
    __syncthreads();

    for (;;) {
        int tok = tok0, at = at0;
#pragma unroll
        for (int i = 0; i < kItems; ++i, step(tok, at)) {
            if (tok >= n || s_off[tok] < 0) continue;
            const bool of_v = at >= row;
            const int c = of_v ? at - row : at, h = c / (D / EL);
            const long long e = s_off[tok] + h * a.head_stride + c % (D / EL) * EL;
            char* pool = static_cast<char*>(const_cast<void*>(of_v ? a.vp : a.kp));
            if (E4M3) {
                float inv;
                if (h < kAppendHeads) {
                    inv = s_inv[2 * h + of_v];
                } else {
                    const float* sc = of_v ? a.vs : a.ks;
                    inv = sc ? 1.0f / sc[h] : 1.0f;
                }
                const uint2 lo = quant8(x[i][0], inv), hi = quant8(x[i][V - 1], inv);
                *reinterpret_cast<uint4*>(pool + e) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                *reinterpret_cast<uint4*>(pool + 2 * e) = x[i][0];
            }
        }
        tok0 = tok;
        at0 = at;
        if (!__syncthreads_or(tok0 < n)) break;
        load();
    }
}

template <int D, bool E4M3>
kda_status append(const PagedArgs& a, const void* k, long long k_stride, const void* v,
                  long long v_stride, const int* granted, cudaStream_t s) {
    // tokens of a CTA: its threads' items, but fewer while CTAs are few
    const int per = 2 * a.HKV * (D / 8);                 // 16-byte loads of a token
    const int full = std::min(kAppendTokens,
                              std::max(1, kAppendThreads * kAppendItems / per));
    const int TB = std::max(1, std::min(full, a.T / (2 * paged::sm_count())));
    TimedLaunch tl("paged_append", s);
    append_kernel<D, E4M3><<<(unsigned)((a.T + TB - 1) / TB), kAppendThreads, 0, s>>>(
        a, TB, static_cast<const __nv_bfloat16*>(k), k_stride,
        static_cast<const __nv_bfloat16*>(v), v_stride, granted);
    return launch_status();
}

}  // namespace

kda_status paged_append_launch(const PagedArgs& a, int D, bool e4m3, const void* k,
                               long long k_stride, const void* v, long long v_stride,
                               const int* granted, cudaStream_t s) {
    if (D == 128)
        return e4m3 ? append<128, true>(a, k, k_stride, v, v_stride, granted, s)
                    : append<128, false>(a, k, k_stride, v, v_stride, granted, s);
    return e4m3 ? append<64, true>(a, k, k_stride, v, v_stride, granted, s)
                : append<64, false>(a, k, k_stride, v, v_stride, granted, s);
}

int* paged_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace kda
