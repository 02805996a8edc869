// Paged key-value cache: appending tokens, and attention over the pages.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_paged_error = 0;   // a kda_status

namespace {

__device__ __forceinline__ void record() { atomicCAS(&g_paged_error, 0, (int)KDA_ERR_SHAPE); }

// The sequence that owns packed token t, or -1 if cu does not rise from 0 to T
// or t lies outside.  All lanes of a warp call it with the same t.
__device__ __forceinline__ int find_seq(const int* __restrict__ cu, int S, int T, int t) {
    const int lane = threadIdx.x & 31;
    bool bad = lane == 0 && (cu[0] != 0 || cu[S] != T);
    int at = -1;
    for (int i = lane; i < S; i += 32) {
        const int a = cu[i], b = cu[i + 1];
        bad |= a > b || a < 0;
        if (a <= t && t < b) at = i;
    }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) at = max(at, __shfl_xor_sync(0xffffffffu, at, o));
    if (bad) {
        if (lane == 0) record();
        return -1;
    }
    return at;
}

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

// One warp per (token, key head) row pair; D / 8 lanes hold eight elements each
// of K, then of V.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256)
append_kernel(const PagedArgs a, const __nv_bfloat16* __restrict__ k, long long k_stride,
              const __nv_bfloat16* __restrict__ v, long long v_stride) {
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = w / a.HKV, h = w % a.HKV;
    if (t >= a.T) return;
    const int s = a.cu ? find_seq(a.cu, a.S, a.T, t) : t;
    if (s < 0) return;
    const int pos = seq_len(a, s) - (a.cu ? a.cu[s + 1] - t : 1);
    if (pos < 0) return;
    const int page = a.table[(size_t)s * a.max_pages + (pos >> a.page_shift)];
    if ((unsigned)page >= (unsigned)a.num_pages) {
        record();
        return;
    }
    const long long off = page * a.page_stride +
                          (pos & ((1 << a.page_shift) - 1)) * a.token_stride + h * a.head_stride;
    const int which = lane / (D / 8), c = lane % (D / 8) * 8;
    if (which > 1) return;
    const __nv_bfloat16* src = (which ? v + t * v_stride : k + t * k_stride) + (long long)h * D + c;
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    char* pool = static_cast<char*>(const_cast<void*>(which ? a.vp : a.kp));
    if (E4M3) {
        const float* sc = which ? a.vs : a.ks;
        *reinterpret_cast<uint2*>(pool + off + c) = quant8(x, sc ? 1.0f / sc[h] : 1.0f);
    } else {
        *reinterpret_cast<uint4*>(pool + 2 * (off + c)) = x;
    }
}

template <bool E4M3>
__device__ __forceinline__ float load_elem(const void* p, long long i) {
    if (E4M3) {
        __nv_fp8_e4m3 c;
        c.__x = static_cast<const unsigned char*>(p)[i];
        return static_cast<float>(c);
    }
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// One warp per query row (token, head): the visible tokens in turn, with the
// running maximum and sum of the softmax; a lane holds D / 32 channels.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) attend_kernel(const PagedArgs a) {
    constexpr int E = D / 32;
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = w / a.HQ, hq = w % a.HQ, h = hq / a.G;
    if (t >= a.T) return;
    const int s = a.cu ? find_seq(a.cu, a.S, a.T, t) : t;
    if (s < 0) return;
    const int p = seq_len(a, s) - (a.cu ? a.cu[s + 1] - t : 1);
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = a.scale * __bfloat162float(a.q[t * a.q_stride + (long long)hq * D + lane * E + e]);
        o[e] = 0.f;
    }
    if (E4M3 && a.ks)
        for (int e = 0; e < E; ++e) q[e] *= a.ks[h];
    const int low = a.window ? max(0, p - a.window + 1) : 0;
    int j = low > 0 && a.sinks > 0 ? 0 : low;
    for (; j <= p; ++j) {
        if (j == a.sinks && j < low) j = low;
        const int page = a.table[(size_t)s * a.max_pages + (j >> a.page_shift)];
        float x = 0.f, v[E] = {};
        if ((unsigned)page < (unsigned)a.num_pages) {
            const long long off = page * a.page_stride +
                                  (j & ((1 << a.page_shift) - 1)) * a.token_stride +
                                  h * a.head_stride + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x += q[e] * load_elem<E4M3>(a.kp, off + e);
                v[e] = load_elem<E4M3>(a.vp, off + e);
            }
        } else {
            record();
        }
#pragma unroll
        for (int r = 16; r > 0; r >>= 1) x += __shfl_xor_sync(0xffffffffu, x, r);
        const float top = fmaxf(m, x), keep = expf(m - top), wgt = expf(x - top);
        l = l * keep + wgt;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + wgt * v[e];
        m = top;
    }
    const float inv = (l > 0.f ? 1.f / l : 0.f) * (E4M3 && a.vs ? a.vs[h] : 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.o[((long long)t * a.HQ + hq) * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
    if (a.lse && lane == 0) a.lse[(long long)t * a.HQ + hq] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <int D, bool E4M3>
kda_status attend(const PagedArgs& a, const char* name, cudaStream_t s) {
    TimedLaunch tl(name, s);
    const long long rows = (long long)a.T * a.HQ;
    attend_kernel<D, E4M3><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a);
    return launch_status();
}

kda_status attend_any(const PagedArgs& a, int D, bool e4m3, const char* name, cudaStream_t s) {
    if (D == 128) return e4m3 ? attend<128, true>(a, name, s) : attend<128, false>(a, name, s);
    return e4m3 ? attend<64, true>(a, name, s) : attend<64, false>(a, name, s);
}

}  // namespace

kda_status paged_append_launch(const PagedArgs& a, int D, bool e4m3, const void* k,
                               long long k_stride, const void* v, long long v_stride,
                               cudaStream_t s) {
    TimedLaunch tl("paged_append", s);
    const unsigned grid = (unsigned)(((long long)a.T * a.HKV + 7) / 8);
    auto* kk = static_cast<const __nv_bfloat16*>(k);
    auto* vv = static_cast<const __nv_bfloat16*>(v);
    if (D == 128 && e4m3)
        append_kernel<128, true><<<grid, 256, 0, s>>>(a, kk, k_stride, vv, v_stride);
    else if (D == 128)
        append_kernel<128, false><<<grid, 256, 0, s>>>(a, kk, k_stride, vv, v_stride);
    else if (e4m3)
        append_kernel<64, true><<<grid, 256, 0, s>>>(a, kk, k_stride, vv, v_stride);
    else
        append_kernel<64, false><<<grid, 256, 0, s>>>(a, kk, k_stride, vv, v_stride);
    return launch_status();
}

size_t paged_prefill_ws_bytes(const PagedArgs& a, int D, bool e4m3) {
    return e4m3 ? 0 : paged_prefill_tc_ws_bytes(a, D);
}
kda_status paged_prefill_launch(const PagedArgs& a, int D, bool e4m3, void* ws, cudaStream_t s) {
    return e4m3 ? attend_any(a, D, true, "paged_prefill", s) : paged_prefill_tc_launch(a, D, ws, s);
}

kda_status paged_take_error(cudaStream_t s) {
    int err = 0;
    if (cudaMemcpyFromSymbolAsync(&err, g_paged_error, sizeof(int), 0, cudaMemcpyDeviceToHost,
                                  s) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return KDA_ERR_CUDA;
    if (err == 0) return KDA_OK;
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_paged_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    cudaStreamSynchronize(s);
    return static_cast<kda_status>(err);
}

}  // namespace kda
