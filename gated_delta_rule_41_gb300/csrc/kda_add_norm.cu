// The residual sum with the norm before the next block, forward and backward:
//
//     r' = r + alpha x,  y = w n,  n = r' / sqrt(mean(r'^2) + eps)
//     dr = dr' + (dn - n mean(dn n)) / sqrt(mean(r'^2) + eps),  dn = dy w
//     dx = alpha dr,  dw = sum over rows of dy n,  dalpha = sum over rows of dr x
//
// One pass over the data, a row in the registers of its threads, as in the gated norm.  The
// forward pass norms r' as summed, before it is rounded to the residual stream's type.
#include "kda_block.cuh"
#include "kda_timing.cuh"

namespace kda {
namespace {

using namespace block;

// R: type of the residual stream (r, r', dr', dr); T: of x, y, dy, dx.

// A thread's part of a row as it lies in memory: r and x, and backward dr' and dy.
template <typename R, typename T, int E, int NC, bool BWD>
struct Row {
    Chunk<R, E> r[NC], u[BWD ? NC : 1];
    Chunk<T, E> x[NC], y[BWD ? NC : 1];

    template <int TPR>
    __device__ __forceinline__ void load(const AddArgs& a, int row, int lane) {
        const R* rp = static_cast<const R*>(a.r) + row * a.r_stride;
        const T* xp = static_cast<const T*>(a.x) + row * a.x_stride;
        const bool with_x = BWD ? a.da != nullptr : a.x != nullptr;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            const bool in = row < a.T && c < a.D;
            const long long e = (long long)row * a.D + c;
            r[i].zero();
            x[i].zero();
            if (in) r[i].load(rp + c);
            if (in && with_x) x[i].load(xp + c);
            if constexpr (BWD) {
                u[i].zero();
                y[i].zero();
                if (in) y[i].load(static_cast<const T*>(a.dy) + e);
                if (in && a.dr) u[i].load(static_cast<const R*>(a.dr) + e);
            }
        }
    }
};

// alpha of a chunk's columns
template <int E>
__device__ __forceinline__ void alphas(const AddArgs& a, int c, float (&v)[E]) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = a.alpha;
    if (a.av.p && c < a.D) a.av.get(c, v);
}

template <typename R, typename T, int E, int TPR, int NC>
__global__ void __launch_bounds__(Rows<TPR>::kThreads) add_fwd_kernel(const AddArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    constexpr bool kAhead = NC <= 2;   // the next row on its way while this one is worked on
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    int turn = 0;
    Row<R, T, E, NC, false> cur, ahead;
    cur.template load<TPR>(a, blockIdx.x * RPC + group, lane);
    for (int row0 = blockIdx.x * RPC; row0 < a.T; row0 += step, ++turn) {
        const int row = row0 + group;
        if constexpr (kAhead) ahead.template load<TPR>(a, row + step, lane);
        float v[NC][E];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            cur.r[i].get(v[i]);
            if (a.x) {
                float f[E], al[E];
                cur.x[i].get(f);
                alphas(a, (i * TPR + lane) * E, al);
#pragma unroll
                for (int j = 0; j < E; ++j) v[i][j] = fmaf(al[j], f[j], v[i][j]);
            }
#pragma unroll
            for (int j = 0; j < E; ++j) sum.x = fmaf(v[i][j], v[i][j], sum.x);
        }
        if constexpr (!kAhead) cur.template load<TPR>(a, row + step, lane);
        sum = row_sum<TPR>(sum, red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            if (row >= a.T || c >= a.D) continue;
            const long long e = (long long)row * a.D + c;
            if (a.r_out) Chunk<R, E>::store(static_cast<R*>(a.r_out) + e, v[i]);
            float w[E];
            a.w.get(c, w);
#pragma unroll
            for (int j = 0; j < E; ++j) v[i][j] *= inv * w[j];
            Chunk<T, E>::store(static_cast<T*>(a.y) + e, v[i]);
        }
        if constexpr (kAhead) cur = ahead;
    }
}

template <typename R, typename T, int E, int TPR, int NC>
__global__ void __launch_bounds__(Rows<TPR>::kThreads) add_bwd_kernel(const AddArgs a) {
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    constexpr bool kAhead = NC <= 2;
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    float dw[NC][E] = {}, da[NC][E] = {};
    int turn = 0;
    Row<R, T, E, NC, true> cur, ahead;
    cur.template load<TPR>(a, blockIdx.x * RPC + group, lane);
    for (int row0 = blockIdx.x * RPC; row0 < a.T; row0 += step, ++turn) {
        const int row = row0 + group;
        if constexpr (kAhead) ahead.template load<TPR>(a, row + step, lane);
        float2 sum = make_float2(0.f, 0.f);   // of r^2 and of dn r
        float w[NC][E];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            float v[E], y[E];
            cur.r[i].get(v);
            cur.y[i].get(y);
#pragma unroll
            for (int j = 0; j < E; ++j) w[i][j] = 0.f;
            if (c < a.D) a.w.get(c, w[i]);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                sum.x = fmaf(v[j], v[j], sum.x);
                sum.y = fmaf(y[j] * w[i][j], v[j], sum.y);
            }
        }
        sum = row_sum<TPR>(sum, red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
        const float m = inv * inv * sum.y * inv_d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            if (row >= a.T || c >= a.D) continue;
            const long long e = (long long)row * a.D + c;
            float v[E], y[E], u[E], f[E], d[E], dx[E];
            cur.r[i].get(v);
            cur.y[i].get(y);
            cur.u[i].get(u);
            cur.x[i].get(f);
            alphas(a, c, dx);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                d[j] = fmaf(inv, fmaf(-m, v[j], y[j] * w[i][j]), u[j]);
                dw[i][j] = fmaf(y[j], v[j] * inv, dw[i][j]);
                da[i][j] = fmaf(d[j], f[j], da[i][j]);
                dx[j] *= d[j];
            }
            Chunk<R, E>::store(static_cast<R*>(a.dres) + e, d);
            if (a.dx) Chunk<T, E>::store(static_cast<T*>(a.dx) + e, dx);
        }
        if constexpr (kAhead)
            cur = ahead;
        else
            cur.template load<TPR>(a, row + step, lane);
    }
    const long long P = gridDim.x;
    if (a.dw) store_part<E, TPR, NC>(dw, a.part + blockIdx.x * (long long)a.D, a.D);
    if (a.da) store_part<E, TPR, NC>(da, a.part + (P + blockIdx.x) * a.D, a.D);
}

template <int E, int TPR, int NC>
struct Fwd {
    template <typename R, typename T>
    static kda_status go(const AddArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, RPC = Rows<TPR>::kRows;
        auto* k = add_fwd_kernel<R, T, E, TPR, NC>;
        static const int per_sm = resident(k, N);
        const int grid = grid_of(per_sm, (a.T + RPC - 1) / RPC);
        TimedLaunch tl("add_norm_fwd", s);
        k<<<grid, N, 0, s>>>(a);
        return launch_status();
    }
    static kda_status run(const AddArgs& a, int type, cudaStream_t s) {
        if (type == 0) return go<__nv_bfloat16, __nv_bfloat16>(a, s);
        return type == 1 ? go<float, float>(a, s) : go<float, __nv_bfloat16>(a, s);
    }
};

template <int E, int TPR, int NC>
struct Bwd {
    template <typename R, typename T>
    static kda_status go(const AddArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, RPC = Rows<TPR>::kRows;
        auto* k = add_bwd_kernel<R, T, E, TPR, NC>;
        static const int per_sm = resident(k, N);
        const int grid = std::min(grid_of(per_sm, (a.T + RPC - 1) / RPC), kPartsPerSm * sm_count());
        {
            TimedLaunch tl("add_norm_bwd", s);
            k<<<grid, N, 0, s>>>(a);
        }
        const kda_status st = launch_status();
        if (st != KDA_OK || (!a.dw && !a.da)) return st;
        return sum_parts_launch(a.part, grid, a.D, a.dw, a.da, s);
    }
    static kda_status run(const AddArgs& a, int type, cudaStream_t s) {
        if (type == 0) return go<__nv_bfloat16, __nv_bfloat16>(a, s);
        return type == 1 ? go<float, float>(a, s) : go<float, __nv_bfloat16>(a, s);
    }
};

bool wide(const AddArgs& a) {
    return a.D % 8 == 0 && a.r_stride % 8 == 0 && a.x_stride % 8 == 0 &&
           aligned16({a.r, a.x, a.r_out, a.y, a.dy, a.dr, a.dres, a.dx, a.av.p, a.w.p});
}

}  // namespace

size_t add_norm_ws_bytes(int T, int D) {
    return align256(2 * (size_t)parts_bound(T) * D * sizeof(float));
}

kda_status add_norm_fwd_launch(const AddArgs& a, int type, cudaStream_t s) {
    return by_width<Fwd, false>(wide(a), a.D, a, type, s);
}

kda_status add_norm_bwd_launch(const AddArgs& a, int type, cudaStream_t s) {
    return by_width<Bwd, true>(wide(a), a.D, a, type, s);
}

}  // namespace kda
