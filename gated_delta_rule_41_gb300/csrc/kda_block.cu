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

// Two threads per block of 32, 16 elements each: rows of D % 32 == 0 elements, 16-byte accesses.
// A pass bounded by HBM.
template <typename T>
__global__ void __launch_bounds__(256) pack_wide_kernel(const T* __restrict__ x, long long rows, int D,
                                                        long long stride, uint8_t* codes,
                                                        uint8_t* scales) {
    const long long per = D / 16, n = rows * per;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i - threadIdx.x < n; i += gridDim.x * 256ll) {
        const bool in = i < n;
        const long long row = rows == 1 ? 0 : i / per, at = i - row * per;
        Chunk<T, 8> r[2];
        r[0].zero();
        r[1].zero();
        if (in) {
            r[0].load(x + row * stride + at * 16);
            r[1].load(x + row * stride + at * 16 + 8);
        }
        float v[2][8];
        r[0].get(v[0]);
        r[1].get(v[1]);
        float top = largest(v[1], largest(v[0]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        if (top > kMaxFloat) {   // in both threads of the block
            top = largest_finite(v[1], largest_finite(v[0]));
            top = fmaxf(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
        }
        if (!in) continue;
        const uint32_t b = scale_byte(top);
        const float inv = inverse_of(b);
        if (b == kTopScale) {
            below_top(v[0]);
            below_top(v[1]);
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = code2(v[j / 2][j % 2 * 4], v[j / 2][j % 2 * 4 + 1], inv) |
                   code2(v[j / 2][j % 2 * 4 + 2], v[j / 2][j % 2 * 4 + 3], inv) << 16;
        reinterpret_cast<uint4*>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        if ((i & 1) == 0) scales[i / 2] = (uint8_t)b;
    }
}

// A warp per block, a lane per element: any width, stride and alignment.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const T* __restrict__ x, long long rows, int D,
                                                   long long stride, uint8_t* codes,
                                                   uint8_t* scales) {
    const int lane = threadIdx.x & 31, per = (D + kScaleBlock - 1) / kScaleBlock;
    const long long n = rows * per;
    for (long long i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < n; i += gridDim.x * 8ll) {
        const long long row = i / per;
        const int c = (int)(i - row * per) * kScaleBlock + lane;
        float v[1] = {c < D ? to_f<T>(x[row * stride + c]) : 0.f};
        float top = largest_finite(v);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        const uint32_t b = scale_byte(top);
        if (b == kTopScale) below_top(v);
        if (c < D) Codes<1>::store(codes + row * D + c, v, inverse_of(b));
        if (lane == 0) scales[i] = (uint8_t)b;
    }
}

// E neighbouring elements of the whole array per thread, which may lie in several blocks and rows.
template <typename T, int E>
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* __restrict__ codes,
                                                     const uint8_t* __restrict__ scales, long long rows,
                                                     int D, T* x) {
    const long long n = rows * D;
    const int per = (D + kScaleBlock - 1) / kScaleBlock;
    for (long long i = (blockIdx.x * 256ll + threadIdx.x) * E; i < n; i += gridDim.x * 256ll * E) {
        const long long row = i / D;
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
        const uint32_t first = r.s;
        r.s = 127;
        float v[E];
        r.get(v);
        uint32_t b = first;
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

int grid_all(long long ctas) { return (int)std::min<long long>(ctas, 8ll * sm_count()); }

template <typename T>
kda_status pack(const void* x, long long rows, int D, long long stride, uint8_t* codes,
                uint8_t* scales, cudaStream_t s) {
    const T* p = static_cast<const T*>(x);
    TimedLaunch tl("pack8", s);
    if (D % kScaleBlock == 0 && stride % 8 == 0 && aligned16({x, codes}))
        pack_wide_kernel<T><<<grid_all((rows * (D / 16) + 255) / 256), 256, 0, s>>>(p, rows, D, stride,
                                                                                  codes, scales);
    else
        pack_kernel<T><<<grid_all((rows * ((D + 31) / 32) + 7) / 8), 256, 0, s>>>(p, rows, D, stride,
                                                                                codes, scales);
    return launch_status();
}

template <typename T>
kda_status unpack(const uint8_t* codes, const uint8_t* scales, long long rows, int D, void* x,
                  cudaStream_t s) {
    T* p = static_cast<T*>(x);
    const long long n = rows * D;
    TimedLaunch tl("unpack8", s);
    if (aligned16({codes, x}))
        unpack_kernel<T, 8><<<grid_all((n + 2047) / 2048), 256, 0, s>>>(codes, scales, rows, D, p);
    else
        unpack_kernel<T, 1><<<grid_all((n + 255) / 256), 256, 0, s>>>(codes, scales, rows, D, p);
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
