// Activations in 8 bits, and the column sums of the norms' backward passes.
#include "kda_block.cuh"
#include "kda_timing.cuh"

namespace kda {

namespace {

using namespace block;

// ---- column sums ----

// One warp-wide strip of 32 columns per CTA, its 32 warps on every 32nd row.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* part, int P, int D, float* out0,
                                                         float* out1) {
    __shared__ float s[32][33];
    float* out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* p = part + (blockIdx.y ? (long long)P * D : 0);
    float v = 0.f;
    if (c < D)
        for (int i = warp; i < P; i += 32) v += p[(long long)i * D + c];
    s[warp][lane] = v;
    __syncthreads();
    // warp w adds up column w
    v = s[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if (lane == 0 && blockIdx.x * 32 + warp < D) out[blockIdx.x * 32 + warp] = v;
}

// ---- 8 bits ----

// 16 neighbouring elements.
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[2][8]) {
    Chunk<__nv_bfloat16, 8> r[2];
    r[0].load(p);
    r[1].load(p + 8);
    r[0].get(v[0]);
    r[1].get(v[1]);
}
__device__ __forceinline__ void load16(const float* p, float (&v)[2][8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 r = __ldcs(reinterpret_cast<const float4*>(p) + j);
        float* o = v[j / 2] + j % 2 * 4;
        o[0] = r.x, o[1] = r.y, o[2] = r.z, o[3] = r.w;
    }
}
// Two threads per block of 32, 16 elements each, one item a thread: rows of D % 32 == 0 elements,
// 16-byte accesses.  A pass bounded by HBM: 32768 x 2048 bf16 34 us, 6.1 TB/s (38 us with a grid that
// walks, eight CTAs per SM and two items on their way; 47 us with four items).
template <typename T>
__global__ void __launch_bounds__(256) pack_wide_kernel(const T* __restrict__ x, long long rows, int D,
                                                        long long stride, uint8_t* codes,
                                                        uint8_t* scales) {
    const long long per = D / 16, n = rows * per, i = blockIdx.x * 256ll + threadIdx.x;
    const long long row = rows == 1 || i >= n ? 0 : i / per;
    float v[2][8] = {};
    if (i < n) load16(x + row * stride + (i - row * per) * 16, v);
    float top = largest(v[1], largest(v[0]));
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    if (top > kMaxFloat) {   // in both threads of the block
        top = largest_finite(v[1], largest_finite(v[0]));
        top = fmaxf(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
    }
    if (i >= n) return;
    const uint32_t b = scale_byte(top);
    const float inv = inverse_of(b);
    if (b == kTopScale) {
        below_top(v[0]);
        below_top(v[1]);
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = code2(v[j / 2][j % 2 * 4], v[j / 2][j % 2 * 4 + 1], inv) |
               code2(v[j / 2][j % 2 * 4 + 2], v[j / 2][j % 2 * 4 + 3], inv) << 16;
    reinterpret_cast<uint4*>(codes)[i] = make_uint4(c[0], c[1], c[2], c[3]);
    if ((i & 1) == 0) scales[i / 2] = (uint8_t)b;
}

// A warp per block, a lane per element, four blocks on their way: any width, stride and alignment.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const T* __restrict__ x, long long rows, int D, int per,
                                                   long long stride, uint8_t* codes,
                                                   uint8_t* scales) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const long long n = rows * per;
    for (long long i0 = (blockIdx.x * 8ll + (threadIdx.x >> 5)) * U; i0 < n; i0 += gridDim.x * 8ll * U) {
        long long row = n <= 0x7fffffff ? (unsigned)i0 / (unsigned)per : i0 / per;
        int block = (int)(i0 - row * per);
        float v[U][1];
        long long at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = block * kScaleBlock + lane;
            const bool in = i0 + u < n && c < D;
            at[u] = in ? row * D + c : -1;
            v[u][0] = in ? to_f<T>(x[row * stride + c]) : 0.f;
            if (++block == per) block = 0, ++row;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float top = largest_finite(v[u]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const uint32_t b = scale_byte(top);
            if (b == kTopScale) below_top(v[u]);
            if (at[u] >= 0) Codes<1>::store(codes + at[u], v[u], inverse_of(b));
            if (lane == 0 && i0 + u < n) scales[i0 + u] = (uint8_t)b;
        }
    }
}

// 16 bytes of values per thread, of one block: D % 32 == 0.
template <typename T>
__global__ void __launch_bounds__(256) unpack_wide_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, long long n,
                                                          T* x) {
    constexpr int E = 16 / sizeof(T);
    const long long i = (blockIdx.x * 256ll + threadIdx.x) * E;
    if (i >= n) return;
    Codes<E> r;
    float v[E];
    r.load(codes + i, scales + i / kScaleBlock);
    r.get(v);
    Chunk<T, E>::store(x + i, v);
}

// E neighbouring elements of the whole array per thread, which may lie in several blocks and rows.
template <typename T, int E>
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales, long long rows,
                                                     int D, int per, T* x) {
    const long long n = rows * D;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) * E; i < n; i += gridDim.x * 256ll * E) {
        const long long row = n <= 0x7fffffff ? (unsigned)i / (unsigned)D : i / D;
        int c = (int)(i - row * D);
        const uint8_t* s = scales + row * per;
        if (E > 1 && i + E > n) {
            // the array's end
            for (long long k = i; k < n; ++k) {
                float v, unused;
                values2(codes[k], v, unused);
                x[k] = from_f<T>(v * scale_of(s[c / kScaleBlock]));
                if (++c == D) c = 0, s += per;
            }
            continue;
        }
        Codes<E> r;
        r.load(codes + i, s + c / kScaleBlock);
        uint32_t b = r.s;
        r.s = 127;
        float v[E];
        r.get(v);
#pragma unroll
        for (int k = 0; k < E; ++k) {
            v[k] *= scale_of(b);
            if (k + 1 < E) {
                ++c;
                if (c == D) {
                    c = 0;
                    s += per;
                    b = *s;
                } else if (c % kScaleBlock == 0) {
                    b = s[c / kScaleBlock];
                }
            }
        }
        Chunk<T, E>::store(x + i, v);
    }
}

// Blocks of a row of D elements, of any D that an int holds.  (The kernels get it as an argument.)
int blocks_of(int D) { return (D - 1) / kScaleBlock + 1; }

// CTAs that walk over what there is.  (The wide kernels' grids cover it: at most 2^40 elements, in
// CTAs of 1024 or more.)
int grid_all(long long ctas) { return (int)std::min<long long>(ctas, 8ll * sm_count()); }

template <typename T>
kda_status pack(const void* x, long long rows, int D, long long stride, uint8_t* codes,
                uint8_t* scales, cudaStream_t s) {
    const T* p = static_cast<const T*>(x);
    TimedLaunch tl("pack8", s);
    if (D % kScaleBlock == 0 && stride % 8 == 0 && aligned16({x, codes}))
        pack_wide_kernel<T><<<(unsigned)((rows * (D / 16) + 255) / 256), 256, 0, s>>>(p, rows, D, stride,
                                                                                    codes, scales);
    else
        pack_kernel<T><<<grid_all((rows * blocks_of(D) + 31) / 32), 256, 0, s>>>(
            p, rows, D, blocks_of(D), stride, codes, scales);
    return launch_status();
}

template <typename T>
kda_status unpack(const uint8_t* codes, const uint8_t* scales, long long rows, int D, void* x,
                  cudaStream_t s) {
    T* p = static_cast<T*>(x);
    const long long n = rows * D;
    TimedLaunch tl("unpack8", s);
    if (D % kScaleBlock == 0 && aligned16({codes, x}))
        unpack_wide_kernel<T><<<(unsigned)((n * sizeof(T) / 16 + 255) / 256), 256, 0, s>>>(codes, scales, n, p);
    else if (aligned16({codes, x}))
        unpack_kernel<T, 4><<<grid_all((n + 1023) / 1024), 256, 0, s>>>(codes, scales, rows, D, blocks_of(D), p);
    else
        unpack_kernel<T, 1><<<grid_all((n + 255) / 256), 256, 0, s>>>(codes, scales, rows, D, blocks_of(D), p);
    return launch_status();
}

}  // namespace

kda_status sum_parts_launch(const float* part, int P, int D, float* out0, float* out1,
                            cudaStream_t s) {
    TimedLaunch tl("sum_parts", s);
    sum_parts_kernel<<<dim3((D + 31) / 32, out1 ? 2 : 1), 1024, 0, s>>>(part, P, D, out0, out1);
    return launch_status();
}

kda_status pack8_launch(const void* x, bool bf16, long long rows, int D, long long stride,
                        uint8_t* codes, uint8_t* scales, cudaStream_t s) {
    return bf16 ? pack<__nv_bfloat16>(x, rows, D, stride, codes, scales, s)
                : pack<float>(x, rows, D, stride, codes, scales, s);
}

kda_status unpack8_launch(const uint8_t* codes, const uint8_t* scales, long long rows, int D,
                          void* x, bool bf16, cudaStream_t s) {
    return bf16 ? unpack<__nv_bfloat16>(codes, scales, rows, D, x, s)
                : unpack<float>(codes, scales, rows, D, x, s);
}

}  // namespace kda
