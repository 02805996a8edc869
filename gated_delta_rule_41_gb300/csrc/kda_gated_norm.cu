// The norm of a mixing layer's output with its gate, forward and backward:
//
//     n = x / sqrt(mean(x^2) + eps),  y = n w s(z),  s(z) = sigmoid(z) or z sigmoid(z)
//     dn = dy w s(z),  dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps)
//     dz = dy n w s'(z),  dw = sum over rows of dy n s(z)
//
// One pass over the data: a row stays in the registers of its threads between the sums over it
// and the results.  With r = 1 / sqrt(mean(x^2) + eps) both sums of the backward pass, those of
// x^2 and of dn x, are formed at once: dx = r (dn - x r^2 mean(dn x)).
#include "kda_block.cuh"
#include "kda_timing.cuh"

namespace kda {
namespace {

using namespace block;

// sigmoid(z) and sigmoid(-z) = 1 - sigmoid(z), each from e = exp(-|z|) without a difference, so that
// both keep their digits far from zero.  float32 tensors take the exact exponential and division.
template <typename T>
__device__ __forceinline__ void sigmoids(float z, float& s, float& other) {
    const float e = sizeof(T) == 2 ? __expf(-fabsf(z)) : expf(-fabsf(z));
    const float p = sizeof(T) == 2 ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e), q = e * p;
    s = z < 0.f ? q : p;
    other = z < 0.f ? p : q;
}
// s(z), and with it s'(z)
template <typename T>
__device__ __forceinline__ float gate(float z, int act) {
    float s, other;
    sigmoids<T>(z, s, other);
    return act == KDA_GATE_SILU ? z * s : s;
}
template <typename T>
__device__ __forceinline__ void gate_grad(float z, int act, float& s, float& ds) {
    sigmoids<T>(z, s, ds);
    if (act == KDA_GATE_SILU) {
        ds = s * fmaf(z, ds, 1.f);
        s *= z;
    } else {
        ds *= s;
    }
}

// (token, head) of a thread's rows, stepped without a division.
struct Place {
    int t, h, dt, dh, H;
    __device__ __forceinline__ Place(int row, int step, int heads) : H(heads) {
        t = row / H;
        h = row - t * H;
        dt = step / H;
        dh = step - dt * H;
    }
    __device__ __forceinline__ void next() {
        t += dt;
        h += dh;
        if (h >= H) {
            h -= H;
            ++t;
        }
    }
};

// The codes and the scale of a chunk; the chunks of a block lie in neighbouring lanes.
template <int E>
__device__ __forceinline__ void keep(float (&v)[E], bool in, uint8_t* code, uint8_t* scale,
                                     int at) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, finite_abs(v[j]));
    if (!in) top = 0.f;
#pragma unroll
    for (int d = kScaleBlock / E / 2; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
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
        const long long e = (long long)row * a.D, b = (long long)row * ((a.D + kScaleBlock - 1) / kScaleBlock);
        const T* xp = static_cast<const T*>(a.x) + at.t * a.x_stride + (long long)at.h * a.D;
        const T* zp = static_cast<const T*>(a.z) + at.t * a.z_stride + (long long)at.h * a.D;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            const bool in = row < rows && c < a.D;
            if constexpr (Q8) {
                xq[i].zero();
                zq[i].zero();
                if (in) {
                    xq[i].load(a.xc + e + c, a.xs + b + c / kScaleBlock);
                    zq[i].load(a.zc + e + c, a.zs + b + c / kScaleBlock);
                }
            } else {
                x[i].zero();
                z[i].zero();
                if (in) {
                    x[i].load(xp + c);
                    z[i].load(zp + c);
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

template <typename T, int E, int TPR, int NC, bool KEEP>
__global__ void __launch_bounds__(Rows<TPR>::kThreads) gated_fwd_kernel(const GatedArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    constexpr bool kAhead = NC <= 2;   // the next row on its way while this one is worked on
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int rows = a.T * a.H, step = gridDim.x * RPC, nblk = (a.D + kScaleBlock - 1) / kScaleBlock;
    const float inv_d = 1.f / a.D;
    Place at(blockIdx.x * RPC + group, step, a.H);
    int turn = 0;
    Row<T, E, NC, false, false> r, ahead;
    r.template load<TPR>(a, at, blockIdx.x * RPC + group, rows, lane);
    for (int row0 = blockIdx.x * RPC; row0 < rows; row0 += step, ++turn) {
        const int row = row0 + group;
        at.next();
        if constexpr (kAhead) ahead.template load<TPR>(a, at, row + step, rows, lane);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float v[E];
            r.get_x(i, v);
#pragma unroll
            for (int j = 0; j < E; ++j) sum.x = fmaf(v[j], v[j], sum.x);
        }
        sum = row_sum<TPR>(sum, red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            const bool in = row < rows && c < a.D;
            float v[E], g[E], w[E], y[E];
            r.get_x(i, v);
            r.get_z(i, g);
            if (in) {
                a.w.get(c, w);
#pragma unroll
                for (int j = 0; j < E; ++j) y[j] = v[j] * inv * w[j] * gate<T>(g[j], a.act);
                Chunk<T, E>::store(static_cast<T*>(a.y) + (long long)row * a.D + c, y);
            }
            if (KEEP) {
                const long long e = (long long)row * a.D, b = (long long)row * nblk;
                keep<E>(v, in, a.xc + e, a.xs + b, c);
                keep<E>(g, in, a.zc + e, a.zs + b, c);
            }
        }
        if constexpr (kAhead)
            r = ahead;
        else
            r.template load<TPR>(a, at, row + step, rows, lane);
    }
}

template <typename T, int E, int TPR, int NC, bool Q8>
__global__ void __launch_bounds__(Rows<TPR>::kThreads) gated_bwd_kernel(const GatedArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    constexpr bool kAhead = NC <= 2;
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int rows = a.T * a.H, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    float dw[NC][E] = {};
    Place at(blockIdx.x * RPC + group, step, a.H);
    int turn = 0;
    Row<T, E, NC, true, Q8> r, ahead;
    r.template load<TPR>(a, at, blockIdx.x * RPC + group, rows, lane);
    for (int row0 = blockIdx.x * RPC; row0 < rows; row0 += step, ++turn) {
        const int row = row0 + group;
        at.next();
        if constexpr (kAhead) ahead.template load<TPR>(a, at, row + step, rows, lane);
        float2 sum = make_float2(0.f, 0.f);   // of x^2 and of dn x
        float s[NC][E], ds[NC][E], w[NC][E];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            float v[E], g[E], y[E];
            r.get_x(i, v);
            r.get_z(i, g);
            r.y[i].get(y);
#pragma unroll
            for (int j = 0; j < E; ++j) w[i][j] = 0.f;
            if (c < a.D) a.w.get(c, w[i]);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                gate_grad<T>(g[j], a.act, s[i][j], ds[i][j]);
                sum.x = fmaf(v[j], v[j], sum.x);
                sum.y = fmaf(y[j] * w[i][j] * s[i][j], v[j], sum.y);
            }
        }
        sum = row_sum<TPR>(sum, red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
        const float m = inv * inv * sum.y * inv_d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            float v[E], y[E], dx[E], dz[E];
            r.get_x(i, v);
            r.y[i].get(y);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float yn = y[j] * v[j] * inv;              // dy n
                dx[j] = inv * fmaf(-m, v[j], y[j] * w[i][j] * s[i][j]);
                dz[j] = yn * w[i][j] * ds[i][j];
                dw[i][j] = fmaf(yn, s[i][j], dw[i][j]);
            }
            if (row < rows && c < a.D) {
                const long long e = (long long)row * a.D + c;
                Chunk<T, E>::store(static_cast<T*>(a.dx) + e, dx);
                Chunk<T, E>::store(static_cast<T*>(a.dz) + e, dz);
            }
        }
        if constexpr (kAhead)
            r = ahead;
        else
            r.template load<TPR>(a, at, row + step, rows, lane);
    }
    if (a.dw) store_part<E, TPR, NC>(dw, a.part + (long long)blockIdx.x * a.D, a.D);
}

template <int E, int TPR, int NC>
struct Fwd {
    template <typename T, bool KEEP>
    static kda_status go(const GatedArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, R = Rows<TPR>::kRows;
        auto* k = gated_fwd_kernel<T, E, TPR, NC, KEEP>;
        static const int per_sm = resident(k, N);
        const int grid = grid_of(per_sm, (a.T * a.H + R - 1) / R);
        TimedLaunch tl("gated_norm_fwd", s);
        k<<<grid, N, 0, s>>>(a);
        return launch_status();
    }
    static kda_status run(const GatedArgs& a, bool bf16, cudaStream_t s) {
        if (a.xc) return bf16 ? go<__nv_bfloat16, true>(a, s) : go<float, true>(a, s);
        return bf16 ? go<__nv_bfloat16, false>(a, s) : go<float, false>(a, s);
    }
};

template <int E, int TPR, int NC>
struct Bwd {
    template <typename T, bool Q8>
    static kda_status go(const GatedArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, R = Rows<TPR>::kRows;
        auto* k = gated_bwd_kernel<T, E, TPR, NC, Q8>;
        static const int per_sm = resident(k, N);
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
        if (a.xs) return bf16 ? go<__nv_bfloat16, true>(a, s) : go<float, true>(a, s);
        return bf16 ? go<__nv_bfloat16, false>(a, s) : go<float, false>(a, s);
    }
};

// 16-byte accesses need widths, strides and pointers that allow them.
bool wide(const GatedArgs& a, bool packed) {
    const int E = 8;
    if (a.D % E || !aligned16({a.x, a.z, a.y, a.dy, a.dx, a.dz, a.xc, a.zc, a.w.p})) return false;
    return packed || (a.x_stride % E == 0 && a.z_stride % E == 0);
}

}  // namespace

size_t gated_norm_ws_bytes(int T, int H, int D) {
    return align256((size_t)parts_bound((long long)T * H) * D * sizeof(float));
}

kda_status gated_norm_fwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s) {
    return by_width<Fwd, false>(wide(a, false), a.D, a, bf16, s);
}

kda_status gated_norm_bwd_launch(const GatedArgs& a, bool bf16, cudaStream_t s) {
    return by_width<Bwd, true>(wide(a, a.xs != nullptr), a.D, a, bf16, s);
}

}  // namespace kda
