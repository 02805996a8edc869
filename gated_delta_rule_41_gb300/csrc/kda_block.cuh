// Shared pieces of the operators around a mixing layer (gated recurrence, gated norm,
// residual sum with norm, 8-bit activations).
#pragma once

#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "kda_paged.cuh"

namespace kda {
namespace block {

constexpr int kScaleBlock = 32;    // neighbours that share a scale
constexpr int kMaxWidth = 16384;   // elements of a row that the norms keep in registers

using paged::sm_count;

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Elementwise arithmetic on a chunk, two at a time where there are two.
template <int E>
__device__ __forceinline__ void vmul(float (&o)[E], const float (&a)[E], const float (&b)[E]) {
    if constexpr (E == 1) {
        o[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 r = __fmul2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]));
            o[j] = r.x, o[j + 1] = r.y;
        }
    }
}
template <int E>
__device__ __forceinline__ void vfma(float (&o)[E], const float (&a)[E], const float (&b)[E],
                                     const float (&c)[E]) {
    if constexpr (E == 1) {
        o[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 r = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]),
                                        make_float2(c[j], c[j + 1]));
            o[j] = r.x, o[j + 1] = r.y;
        }
    }
}
template <int E>
__device__ __forceinline__ void vmul(float (&o)[E], const float (&a)[E], float b) {
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = b;
    vmul(o, a, v);
}
template <int E>
__device__ __forceinline__ void vfma(float (&o)[E], const float (&a)[E], float b, const float (&c)[E]) {
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = b;
    vfma(o, a, v, c);
}
// A running sum of products, kept in two parts.
template <int E>
__device__ __forceinline__ void vdot(float2& sum, const float (&a)[E], const float (&b)[E]) {
    if constexpr (E == 1) {
        sum.x = fmaf(a[0], b[0], sum.x);
    } else {
#pragma unroll
        for (int j = 0; j < E; j += 2)
            sum = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), sum);
    }
}

// E neighbouring elements of type T as they lie in memory: E = 8 for bf16, 4 for float32 and what
// is beside it (16-byte accesses; neighbouring lanes then read whole sectors), 1 for rows that
// allow no more.
template <typename T, int E>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        r = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        unpack2(r.x, v[0], v[1]);
        unpack2(r.y, v[2], v[3]);
        unpack2(r.z, v[4], v[5]);
        unpack2(r.w, v[6], v[7]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]),
                                                  pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
};
template <>
struct Chunk<__nv_bfloat16, 4> {
    uint2 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        r = __ldcs(reinterpret_cast<const uint2*>(p));
    }
    __device__ __forceinline__ void zero() { r = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        unpack2(r.x, v[0], v[1]);
        unpack2(r.y, v[2], v[3]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    }
};
template <>
struct Chunk<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <typename T>
struct Chunk<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = *p; }
    __device__ __forceinline__ void zero() { r = from_f<T>(0.f); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f<T>(r); }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { *p = from_f<T>(v[0]); }
};

// ---- 8-bit blocks: 32 neighbours share the smallest 2^e, e >= -126, with max |x| <= 448 2^e ----

// e + 127 from the largest finite magnitude of a block.  448 = 1.75 * 2^8: with top = m * 2^k,
// 1 <= m < 2, e = k - 8, or k - 7 where m > 1.75; both read from the bits of top (a subnormal top
// has k < -126 and ends at the lower limit).
__device__ __forceinline__ uint32_t scale_byte(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
    return (uint32_t)(max(e, -126) + 127);
}
// 2^e and 2^-e of a scale byte (1..247: both are normal numbers)
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float inverse_of(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}
// The largest magnitude of a chunk: infinite where there is an infinity; NaN do not count.
template <int E>
__device__ __forceinline__ float largest(const float (&v)[E], float top = 0.f) {
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, fabsf(v[j]));
    return top;
}
// With an infinity in the block: the chunk's largest finite magnitude, its infinities made NaN.  (As
// codes they may not pass for finite values in the backward pass; NaN become NaN by themselves.)
constexpr float kMaxFloat = 3.402823466e38f;
template <int E>
__device__ __forceinline__ float largest_finite(float (&v)[E], float top = 0.f) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if (fabsf(v[j]) <= kMaxFloat)
            top = fmaxf(top, fabsf(v[j]));
        else
            v[j] = __uint_as_float(0x7fffffffu);
    }
    return top;
}
// With the largest scale a code of 256 would stand for 2^128: values next to the largest float go
// to the code below it, 240, which is no further off than 2^-4.
constexpr uint32_t kTopScale = 247;
template <int E>
__device__ __forceinline__ void below_top(float (&v)[E]) {
    constexpr float most = 240.f * 1.329227995784916e36f;   // 240 * 2^120
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (fabsf(v[j]) > most) v[j] = copysignf(most, v[j]);
}
// Codes of a pair times the scale's inverse (the lower byte is a's).
__device__ __forceinline__ uint32_t code2(float a, float b, float inv) {
    return __nv_cvt_float2_to_fp8x2(__fmul2_rn(make_float2(a, b), make_float2(inv, inv)), __NV_SATFINITE,
                                    __NV_E4M3);
}
__device__ __forceinline__ void values2(uint32_t two, float& a, float& b) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    a = f.x;
    b = f.y;
}

// E codes as they lie in memory, and the scale of their block.
template <int E>
struct Codes;
template <>
struct Codes<8> {
    uint2 r;
    uint32_t s;
    __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* scale) {
        r = __ldcs(reinterpret_cast<const uint2*>(p));
        s = *scale;
    }
    __device__ __forceinline__ void zero() {
        r = make_uint2(0, 0);
        s = 127;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        values2(r.x & 0xffffu, v[0], v[1]);
        values2(r.x >> 16, v[2], v[3]);
        values2(r.y & 0xffffu, v[4], v[5]);
        values2(r.y >> 16, v[6], v[7]);
        vmul(v, v, scale_of(s));
    }
    static __device__ __forceinline__ void store(uint8_t* p, const float (&v)[8], float inv) {
        *reinterpret_cast<uint2*>(p) =
            make_uint2(code2(v[0], v[1], inv) | code2(v[2], v[3], inv) << 16,
                       code2(v[4], v[5], inv) | code2(v[6], v[7], inv) << 16);
    }
};
template <>
struct Codes<4> {
    uint32_t r, s;
    __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* scale) {
        r = __ldcs(reinterpret_cast<const uint32_t*>(p));
        s = *scale;
    }
    __device__ __forceinline__ void zero() {
        r = 0;
        s = 127;
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        values2(r & 0xffffu, v[0], v[1]);
        values2(r >> 16, v[2], v[3]);
        vmul(v, v, scale_of(s));
    }
    static __device__ __forceinline__ void store(uint8_t* p, const float (&v)[4], float inv) {
        *reinterpret_cast<uint32_t*>(p) = code2(v[0], v[1], inv) | code2(v[2], v[3], inv) << 16;
    }
};
template <>
struct Codes<1> {
    uint8_t r;
    uint32_t s;
    __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* scale) {
        r = *p;
        s = *scale;
    }
    __device__ __forceinline__ void zero() {
        r = 0;
        s = 127;
    }
    __device__ __forceinline__ void get(float (&v)[1]) const {
        float unused;
        values2(r, v[0], unused);
        v[0] *= scale_of(s);
    }
    static __device__ __forceinline__ void store(uint8_t* p, const float (&v)[1], float inv) {
        *p = (uint8_t)code2(v[0], 0.f, inv);
    }
};

// A parameter vector, float32 or bf16; ones where there is none.  Read again for each row: it
// stays in L1, and registers are better spent on rows in flight.
struct Param {
    const void* p;
    bool bf16;
    template <int E>
    __device__ __forceinline__ void get(int c, float (&v)[E]) const {
        if (!p) {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = 1.f;
        } else if constexpr (E == 1) {
            v[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c])
                        : __ldg(static_cast<const float*>(p) + c);
        } else if (bf16) {
            const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                const uint2 r = __ldg(q + j / 4);
                unpack2(r.x, v[j], v[j + 1]);
                unpack2(r.y, v[j + 2], v[j + 3]);
            }
        } else {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
#pragma unroll
            for (int j = 0; j < E; j += 4) {
                const float4 r = __ldg(q + j / 4);
                v[j] = r.x, v[j + 1] = r.y, v[j + 2] = r.z, v[j + 3] = r.w;
            }
        }
    }
};

// Sums over the TPR threads of a row (a power of two), for every thread of it.  Rows of more than
// a warp go through shared memory: `red` has one entry per warp of the CTA for each of two turns,
// so that one barrier a turn is enough.
template <int TPR, bool BOTH>
__device__ __forceinline__ float2 row_sum(float2 v, float2* red, int turn, int warps) {
#pragma unroll
    for (int d = (TPR < 32 ? TPR : 32) / 2; d > 0; d >>= 1) {
        v.x += __shfl_xor_sync(~0u, v.x, d);
        if (BOTH) v.y += __shfl_xor_sync(~0u, v.y, d);
    }
    if (TPR > 32) {
        float2* at = red + (turn & 1) * warps;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) at[warp] = v;
        __syncthreads();
        constexpr int W = TPR > 32 ? TPR / 32 : 1;
        const int first = warp / W * W;
        v = at[first];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            const float2 o = at[first + i];
            v.x += o.x;
            v.y += o.y;
        }
    }
    return v;
}

// Where a thread's rows lie: threads per row, rows per CTA.
template <int TPR>
struct Rows {
    static constexpr int kThreads = TPR > 256 ? TPR : 256;
    static constexpr int kRows = kThreads / TPR;
    // CTAs that an SM has to hold: left to the compiler, but for the widest (it would spill for two)
    static constexpr int kMin = kThreads > 256 ? 1 : 0;
};

// Picks the widths a kernel is made for: a row's elements stay in registers, E * NC of them in
// each of TPR threads.  F: template <int E, int TPR, int NC> struct with a static run(args...).
// E, as chunk_of gives it, is the widest access that widths, strides and pointers allow: one element at a time
// 1000 columns' worth of work takes twice the time (residual norm of 32768 x 1001 104 us, x 1024 52 us),
// 77 columns three times that of 128.  A row has as few threads as hold it in registers, since rows inside
// a warp need no barrier; from 256 E elements on it has a CTA (2048 bf16: 87 us; in one warp, eight
// chunks to a lane, 109 us).
template <template <int, int, int> class F, int E, typename... A>
kda_status by_width(int D, A&&... args) {
    if constexpr (E == 1) {
        if (D <= 128) return F<1, 32, 4>::run(args...);
        if (D <= 512) return F<1, 128, 4>::run(args...);
        if (D <= 2048) return F<1, 256, 8>::run(args...);
        return F<1, 1024, 16>::run(args...);
    } else {
        // (never fewer threads than a block of 32 elements takes)
        if constexpr (4 * E >= kScaleBlock)
            if (D <= 4 * E) return F<E, 4, 1>::run(args...);
        if (D <= 8 * E) return F<E, 8, 1>::run(args...);
        if (D <= 16 * E) return F<E, 16, 1>::run(args...);
        if (D <= 32 * E) return F<E, 32, 1>::run(args...);
        if (D <= 64 * E) return F<E, 32, 2>::run(args...);
        if (D <= 128 * E) return F<E, 64, 2>::run(args...);
        if (D <= 256 * E) return F<E, 256, 1>::run(args...);
        if (D <= 512 * E) return F<E, 256, 2>::run(args...);
        if (D <= 1024 * E) return F<E, 256, 4>::run(args...);
        if constexpr (2048 * E < kMaxWidth)
            if (D > 2048 * E) return F<E, 1024, 4>::run(args...);
        return F<E, 512, 4>::run(args...);
    }
}

inline bool aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15) return false;
    return true;
}

// CTAs of a kernel that walks over its rows: all that an SM holds at once, or fewer.  Shared memory
// is allowed and the CTAs are counted for one device at a time, so both are kept per device.
struct Resident {
    std::atomic<int> n[64] = {};   // 0: not known yet
    template <typename K>
    kda_status get(K kernel, int threads, size_t smem, int& per_sm) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
        per_sm = n[dev].load(std::memory_order_acquire);
        if (per_sm) return KDA_OK;
        // (without the attribute 48 KB, static shared memory included)
        if ((smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      (int)smem) != cudaSuccess) ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess ||
            per_sm < 1) {
            cudaGetLastError();   // said here, not by the next call
            return KDA_ERR_CUDA;
        }
        n[dev].store(per_sm, std::memory_order_release);
        return KDA_OK;
    }
};
inline int grid_of(int per_sm, long long ctas_of_work) {
    return (int)std::min<long long>((long long)per_sm * sm_count(), ctas_of_work);
}

// Column sums over rows: each CTA leaves one row of partial sums in the workspace, and
// sum_parts_launch adds them up in order, so that the same call gives the same bits.
constexpr int kPartsPerSm = 8;
inline int parts_bound(long long rows) {
    return (int)std::min<long long>((long long)kPartsPerSm * sm_count(), rows);
}

// The sums of a CTA's rows into its row of partial sums: the row groups one after the other,
// through shared memory.
template <int E, int TPR, int NC>
__device__ __forceinline__ void store_part(const float (&v)[NC][E], float* part, int D) {
    constexpr int G = Rows<TPR>::kRows;
    __shared__ float sum[G > 1 ? TPR * NC * E : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    for (int g = 0; g < G; ++g) {
        if (G > 1) __syncthreads();
        if (g != group) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = (i * TPR + lane) * E + j, k = G > 1 ? (i * E + j) * TPR + lane : 0;
                float x = v[i][j];
                if (G > 1 && g > 0) x += sum[k];
                if (g == G - 1) {
                    if (c < D) part[c] = x;
                } else {
                    sum[k] = x;
                }
            }
    }
}

}  // namespace block

// Column sums of part [P][D] into out0, and of the [P][D] behind it into out1 (null: left out).
kda_status sum_parts_launch(const float* part, int P, int D, float* out0, float* out1,
                            cudaStream_t s);

// ---- launchers (validated arguments only) ----
struct ScanArgs {
    int B, T, C;
    bool tied;
    long long x_batch, x_token, g_batch, g_token;
    const void *x, *g;
    const float* h0;        // [B or nseq][C], may be null
    const int* cu;          // null: B sequences of T tokens
    int nseq;
    void* o;                // may be null (states alone)
    float *ht, *states;     // may be null
    // backward
    const void* dout;
    const float* dht;
    void *dx, *dg;
    float* dh0;
};
kda_status scan_fwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s);
kda_status scan_bwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s);
kda_status scan_step_launch(int B, int C, bool bf16, bool tied, const void* x, long long x_row,
                            const void* g, long long g_row, const float* state, float* next,
                            void* o, cudaStream_t s);

struct GatedArgs {
    int T, H, D;
    int act;                        // kda_gate
    float eps;
    long long x_stride, z_stride;   // of tokens, in elements
    const void *x, *z;
    block::Param w;
    void* y;
    uint8_t *xc, *xs, *zc, *zs;     // forward: kept codes and scales, or null; backward: inputs
    const void* dy;
    void *dx, *dz;
    float* dw;                      // may be null
    float* part;                    // workspace
};
kda_status gated_norm_fwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s);
kda_status gated_norm_bwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s);
size_t gated_norm_ws_bytes(int T, int H, int D);

struct AddArgs {
    int T, D;
    float eps, alpha;
    long long r_stride, x_stride;
    const void *r, *x;              // x may be null
    block::Param av, w;             // av.p null: alpha
    void *r_out, *y;
    const void *dy, *dr;            // dr may be null
    void *dres, *dx;                // dx may be null
    float *dw, *da;                 // may be null
    float* part;
};
// type: 0 all bf16, 1 all float32, 2 bf16 beside a float32 residual stream
kda_status add_norm_fwd_launch(const AddArgs& a, int type, cudaStream_t s);
kda_status add_norm_bwd_launch(const AddArgs& a, int type, cudaStream_t s);
size_t add_norm_ws_bytes(int T, int D);

kda_status pack8_launch(const void* x, bool bf16, long long rows, int D, long long stride,
                        uint8_t* codes, uint8_t* scales, cudaStream_t s);
kda_status unpack8_launch(const uint8_t* codes, const uint8_t* scales, long long rows, int D,
                          void* x, bool bf16, cudaStream_t s);

}  // namespace kda
