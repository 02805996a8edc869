// The norm of a mixing layer's output with its gate, forward and backward:
//
//     n = x / sqrt(mean(x^2) + eps),  y = n w s(z),  s(z) = sigmoid(z) or z sigmoid(z)
//     dn = dy w s(z),  dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps)
//     dz = dy n w s'(z),  dw = sum over rows of dy n s(z)
//
// One pass over the data, bounded by HBM: a row stays in the registers of its threads between the sums
// over it and the results; 16 threads for 128 elements, so that two rows fill a warp and the sums
// take four shuffles.  32768 x 16 x 128 bf16 on one GB300: forward with 8-bit copies of both inputs
// 88 us, 6.1 TB/s (0.92 of the copy rate), without 64 us; backward from these copies 104 us, 5.2 TB/s
// (0.78; 57 % of the issue slots), from bf16 114 us.  With r = 1 / sqrt(mean(x^2) + eps) both sums of the backward pass, those of
// x^2 and of dn x, are formed at once: dx = r (dn - x r^2 mean(dn x)).
#include "kda_block.cuh"
#include "kda_timing.cuh"

namespace kda {
namespace {

using namespace block;

// Powers of two and reciprocals of bf16 tensors are the fast ones (2^-22 of the result, and the rounding
// of the argument), float32 ones take the exact exponential and division.  The fast ones give 0 below
// 2^-126, where both types have subnormal numbers (and z, or a large x, may lift what is below them), so
// they are kept away from there: exponentials as the square of their root's, sums with both terms times
// 2^-20.  A sigmoid is then right down to 2^-146, and 0 below.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f, kBits = 20.f, kDown = 1.f / (1 << 20);

// exp(-|z|) = e and 1 / (1 + e)
template <typename T>
__device__ __forceinline__ float logistic(float z, float& e) {
    if (sizeof(T) == 2) {
        e = exp2_fast(fabsf(z) * (-kLog2e / 2));
        e *= e;
        return rcp_fast(1.f + e);
    }
    e = expf(-fabsf(z));
    return 1.f / (1.f + e);
}
template <typename T>
__device__ __forceinline__ float gate(float z, int act) {
    float s;
    if (sizeof(T) == 2) {
        // 1 / (1 + exp(-z)), the sum times 2^-20
        s = rcp_fast(kDown + exp2_fast(fmaf(z, -kLog2e, -kBits))) * kDown;
    } else {
        float e;
        s = logistic<T>(z, e);
        if (z < 0.f) s *= e;
    }
    return act == KDA_GATE_SILU ? z * s : s;
}
// s(z) and s'(z).  sigmoid(z) and sigmoid(-z) = 1 - sigmoid(z) come from exp(-|z|) without a
// difference, so that both keep their digits far from zero.
template <typename T>
__device__ __forceinline__ void gate_grad(float z, int act, float& s, float& ds) {
    float e;
    const float p = logistic<T>(z, e), q = e * p;
    s = z < 0.f ? q : p;
    ds = z < 0.f ? p : q;
    if (act == KDA_GATE_SILU) {
        ds = s * fmaf(z, ds, 1.f);
        s *= z;
    } else {
        ds *= s;
    }
}

// (token, head) of a thread's rows, stepped without a division.
struct Place {
    int t, h, dt, dh;
    __device__ __forceinline__ Place(const GatedArgs& a, int row, int step) {
        t = row / a.H;
        h = row - t * a.H;
        dt = step / a.H;
        dh = step - dt * a.H;
    }
    __device__ __forceinline__ void next(const GatedArgs& a) {
        t += dt;
        h += dh;
        if (h >= a.H) {
            h -= a.H;
            ++t;
        }
    }
};

__host__ __device__ __forceinline__ int blocks_of(int D) { return (D + kScaleBlock - 1) / kScaleBlock; }

// The codes and the scale of a chunk; the chunks of a block lie in neighbouring lanes.
template <int E>
__device__ __forceinline__ void keep(float (&v)[E], bool in, uint8_t* code, uint8_t* scale, int at) {
    float top = largest(v);
    if (!in) top = 0.f;
#pragma unroll
    for (int d = kScaleBlock / E / 2; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    if (__any_sync(~0u, top > kMaxFloat)) {
        top = in ? largest_finite(v) : 0.f;
#pragma unroll
        for (int d = kScaleBlock / E / 2; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    }
    if (!in) return;
    const uint32_t b = scale_byte(top);
    if (b == kTopScale) below_top(v);
    Codes<E>::store(code + at, v, inverse_of(b));
    if (at % kScaleBlock == 0) scale[at / kScaleBlock] = (uint8_t)b;
}

// A thread's part of a row as it lies in memory: x, the gate, and backward dy.  Q8: x and the gate
// are codes with scales.
template <typename T, int E, int NC, bool BWD, bool Q8>
struct Row {
    Chunk<T, E> x[Q8 ? 1 : NC], z[Q8 ? 1 : NC], y[BWD ? NC : 1];
    Codes<E> xq[Q8 ? NC : 1], zq[Q8 ? NC : 1];

    template <int TPR>
    __device__ __forceinline__ void load(const GatedArgs& a, const Place& at, int row, int rows, int lane) {
        const long long e = (long long)row * a.D;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            const bool in = row < rows && c < a.D;
            if constexpr (Q8) {
                xq[i].zero();
                zq[i].zero();
                if (in) {
                    const long long b = (long long)row * blocks_of(a.D) + c / kScaleBlock;
                    xq[i].load(a.xc + e + c, a.xs + b);
                    zq[i].load(a.zc + e + c, a.zs + b);
                }
            } else {
                x[i].zero();
                z[i].zero();
                if (in) {
                    const long long h = (long long)at.h * a.D + c;
                    x[i].load(static_cast<const T*>(a.x) + at.t * a.x_stride + h);
                    z[i].load(static_cast<const T*>(a.z) + at.t * a.z_stride + h);
                }
            }
            if constexpr (BWD) {
                y[i].zero();
                if (in) y[i].load(static_cast<const T*>(a.dy) + e + c);
            }
        }
    }
    __device__ __forceinline__ void get_x(int i, float (&v)[E]) const {
        if constexpr (Q8)
            xq[i].get(v);
        else
            x[i].get(v);
    }
    __device__ __forceinline__ void get_z(int i, float (&v)[E]) const {
        if constexpr (Q8)
            zq[i].get(v);
        else
            z[i].get(v);
    }
};

// Rows on their way while one is worked on, in registers: 32 to 48 bytes a thread and row are too
// few in flight with one.  (32768 x 16 x 128 bf16: forward with 8-bit copies 109 us with one and 91
// with three; backward from them 114 us with one at three CTAs per SM, 116 with two and 107 with three at
// two.)
template <int NC, bool BWD>
constexpr int kDepth = NC == 1 ? 3 : NC == 2 && !BWD ? 2 : 1;

template <typename T, int E, int TPR, int NC, bool KEEP>
__global__ void __launch_bounds__(Rows<TPR>::kThreads, Rows<TPR>::kMin) gated_fwd_kernel(const GatedArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32, D = kDepth<NC, false>;
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int rows = a.T * a.H, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    int row = blockIdx.x * RPC + group, turn = 0;
    Place at(a, row, step);   // of the next row to load
    Row<T, E, NC, false, false> ring[D];
#pragma unroll
    for (int k = 0; k < D; ++k, at.next(a)) ring[k].template load<TPR>(a, at, row + k * step, rows, lane);
    float w[NC <= 2 ? NC : 1][E];
    if constexpr (NC <= 2) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if ((i * TPR + lane) * E < a.D) a.w.get((i * TPR + lane) * E, w[i]);
    }
    while (row - group < rows) {
#pragma unroll
        for (int k = 0; k < D; ++k, row += step, ++turn) {
            if (row - group >= rows) break;   // alike in the whole CTA
            float v[NC][E], g[NC][E];
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                ring[k].get_x(i, v[i]);
                ring[k].get_z(i, g[i]);
                vdot(sum, v[i], v[i]);
            }
            ring[k].template load<TPR>(a, at, row + D * step, rows, lane);
            at.next(a);
            sum.x += sum.y;
            sum = row_sum<TPR, false>(sum, red, turn, W);
            const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
            const long long e = (long long)row * a.D, b = (long long)row * blocks_of(a.D);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = (i * TPR + lane) * E;
                const bool in = row < rows && c < a.D;
                if (in) {
                    float f[E], y[E];
                    if constexpr (NC <= 2) {
                        vmul(y, v[i], w[i]);
                    } else {
                        a.w.get(c, f);
                        vmul(y, v[i], f);
                    }
#pragma unroll
                    for (int j = 0; j < E; ++j) f[j] = gate<T>(g[i][j], a.act);
                    vmul(y, y, f);
                    vmul(y, y, inv);
                    Chunk<T, E>::store(static_cast<T*>(a.y) + e + c, y);
                }
                if (KEEP) {
                    keep<E>(v[i], in, a.xc + e, a.xs + b, c);
                    keep<E>(g[i], in, a.zc + e, a.zs + b, c);
                }
            }
        }
    }
}

template <typename T, int E, int TPR, int NC, bool Q8>
__global__ void __launch_bounds__(Rows<TPR>::kThreads, NC == 1 && TPR <= 256 ? 2 : Rows<TPR>::kMin) gated_bwd_kernel(const GatedArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32, D = kDepth<NC, true>;
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int rows = a.T * a.H, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    float dw[NC][E] = {}, w1[E] = {};
    if (NC == 1 && lane * E < a.D) a.w.get(lane * E, w1);
    int row = blockIdx.x * RPC + group, turn = 0;
    Place at(a, row, step);
    Row<T, E, NC, true, Q8> ring[D];
#pragma unroll
    for (int k = 0; k < D; ++k, at.next(a)) ring[k].template load<TPR>(a, at, row + k * step, rows, lane);
    while (row - group < rows) {
#pragma unroll
        for (int k = 0; k < D; ++k, row += step, ++turn) {
            if (row - group >= rows) break;   // alike in the whole CTA
            float2 s2 = make_float2(0.f, 0.f), sn = s2;   // sums of x^2 and of dn x
            float v[NC][E], y[NC][E], s[NC][E], wds[NC][E], dn[NC][E];
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = (i * TPR + lane) * E;
                float g[E], w[E], ds[E];
                ring[k].get_x(i, v[i]);
                ring[k].get_z(i, g);
                ring[k].y[i].get(y[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) w[j] = NC == 1 ? w1[j] : 0.f;
                if (NC > 1 && c < a.D) a.w.get(c, w);
#pragma unroll
                for (int j = 0; j < E; ++j) gate_grad<T>(g[j], a.act, s[i][j], ds[j]);
                vmul(wds[i], w, ds);
                vmul(dn[i], y[i], w);
                vmul(dn[i], dn[i], s[i]);
                vdot(s2, v[i], v[i]);
                vdot(sn, dn[i], v[i]);
            }
            ring[k].template load<TPR>(a, at, row + D * step, rows, lane);
            at.next(a);
            const float2 sum = row_sum<TPR, true>(make_float2(s2.x + s2.y, sn.x + sn.y), red, turn, W);
            const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
            const float m = inv * (inv * (sum.y * inv_d));   // (inv * inv may overflow)
            const long long e = (long long)row * a.D;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = (i * TPR + lane) * E;
                float yn[E];
                vfma(dn[i], v[i], -m, dn[i]);
                vmul(dn[i], dn[i], inv);                 // dx
                vmul(yn, v[i], inv);
                vmul(yn, y[i], yn);                      // dy n
                vfma(dw[i], yn, s[i], dw[i]);
                vmul(yn, yn, wds[i]);                    // dz
                if (row < rows && c < a.D) {
                    Chunk<T, E>::store(static_cast<T*>(a.dx) + e + c, dn[i]);
                    Chunk<T, E>::store(static_cast<T*>(a.dz) + e + c, yn);
                }
            }
        }
    }
    if (a.dw) store_part<E, TPR, NC>(dw, a.part + (long long)blockIdx.x * a.D, a.D);
}

template <int E, int TPR, int NC>
struct Fwd {
    template <typename T, bool KEEP>
    static kda_status go(const GatedArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, R = Rows<TPR>::kRows;
        auto* k = gated_fwd_kernel<T, E, TPR, NC, KEEP>;
        static Resident resident;
        int per_sm = 0;
        if (resident.get(k, N, 0, per_sm) != KDA_OK) return KDA_ERR_CUDA;
        const int grid = grid_of(per_sm, (a.T * a.H + R - 1) / R);
        TimedLaunch tl("gated_norm_fwd", s);
        k<<<grid, N, 0, s>>>(a);
        return launch_status();
    }
    static kda_status run(const GatedArgs& a, bool bf16, cudaStream_t s) {
        if constexpr (E != 8)
            if (!bf16) return a.xc ? go<float, true>(a, s) : go<float, false>(a, s);
        return a.xc ? go<__nv_bfloat16, true>(a, s) : go<__nv_bfloat16, false>(a, s);
    }
};

template <int E, int TPR, int NC>
struct Bwd {
    template <typename T, bool Q8>
    static kda_status go(const GatedArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, R = Rows<TPR>::kRows;
        auto* k = gated_bwd_kernel<T, E, TPR, NC, Q8>;
        static Resident resident;
        int per_sm = 0;
        if (resident.get(k, N, 0, per_sm) != KDA_OK) return KDA_ERR_CUDA;
        const int grid = std::min(grid_of(per_sm, (a.T * a.H + R - 1) / R), kPartsPerSm * sm_count());
        {
            TimedLaunch tl("gated_norm_bwd", s);
            k<<<grid, N, 0, s>>>(a);
        }
        const kda_status st = launch_status();
        if (st != KDA_OK || !a.dw) return st;
        return sum_parts_launch(a.part, grid, a.D, a.dw, nullptr, s);
    }
    static kda_status run(const GatedArgs& a, bool bf16, cudaStream_t s) {
        if constexpr (E != 8)
            if (!bf16) return a.xs ? go<float, true>(a, s) : go<float, false>(a, s);
        return a.xs ? go<__nv_bfloat16, true>(a, s) : go<__nv_bfloat16, false>(a, s);
    }
};

// Elements of an access: 8 of bf16 or 4 where widths, strides and pointers allow them.
int chunk_of(const GatedArgs& a, bool bf16, bool packed) {
    if (!aligned16({a.x, a.z, a.y, a.dy, a.dx, a.dz, a.xc, a.zc, a.w.p})) return 1;
    for (int E = bf16 ? 8 : 4; E >= 4; E /= 2)
        if (a.D % E == 0 && (packed || (a.x_stride % E == 0 && a.z_stride % E == 0))) return E;
    return 1;
}
template <template <int, int, int> class F>
kda_status launch(const GatedArgs& a, bool bf16, bool packed, cudaStream_t s) {
    const int E = chunk_of(a, bf16, packed);
    if (E == 8) return by_width<F, 8>(a.D, a, bf16, s);
    return E == 4 ? by_width<F, 4>(a.D, a, bf16, s) : by_width<F, 1>(a.D, a, bf16, s);
}

}  // namespace

size_t gated_norm_ws_bytes(int T, int H, int D) {
    return align256((size_t)parts_bound((long long)T * H) * D * sizeof(float));
}

kda_status gated_norm_fwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s) {
    return launch<Fwd>(a, bf16, false, s);
}

kda_status gated_norm_bwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s) {
    return launch<Bwd>(a, bf16, a.xs != nullptr, s);
}

}  // namespace kda
