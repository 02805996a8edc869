// Paged key-value cache: appending tokens.
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
