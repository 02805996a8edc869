// The residual sum with the norm before the next block, forward and backward:
//
//     r' = r + alpha x,  y = w n,  n = r' / sqrt(mean(r'^2) + eps)
//     dr = dr' + (dn - n mean(dn n)) / sqrt(mean(r'^2) + eps),  dn = dy w
//     dx = alpha dr,  dw = sum over rows of dy n,  dalpha = sum over rows of dr x
//
// One pass over the data, bounded by HBM, a row in the registers of its threads, as in the gated
// norm.  One GB300: forward of 32768 x 2048 bf16 85 us, 6.3 TB/s (0.94 of the copy rate); backward of 20011
// x 2048 with a float32 stream 128 us, 5.8 TB/s (0.86).  The
// forward pass norms r' as summed, before it is rounded to the residual stream's type.
#include "kda_block.cuh"
#include "kda_ptx.cuh"
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
};

// Rows on their way while one is worked on.  Wide rows go through shared memory, each thread by
// asynchronous copies into slots of its own (no barrier, no registers): with the next row in
// registers alone, the backward pass of 20011 x 2048 had too few bytes in flight (148 us).
// Others are loaded where they are used.
template <typename R, typename T, int E, int TPR, int NC, bool BWD>
struct Feed {
    static constexpr int kThreads = Rows<TPR>::kThreads;
    // bytes of a thread's chunk of each type, and of its part of a row
    static constexpr int kR = sizeof(Chunk<R, E>), kT = sizeof(Chunk<T, E>);
    static constexpr int kStage = NC * (kR + kT) * (BWD ? 2 : 1) * kThreads;
    // slots: four as long as two CTAs then fit an SM, or as many as fit; the widest rows have none
    static constexpr int kSlots = E == 1                     ? 1
                                  : kStage * 4 <= 100 * 1024 ? 4
                                  : kStage * 3 <= 100 * 1024 ? 3
                                  : kStage * 2 <= 200 * 1024 ? 2
                                                             : 1;
    static constexpr bool kRing = kSlots > 1;
    // rows begun before they are used: a slot is filled again one turn after it was read
    static constexpr int kAhead = kSlots - 1;
    static constexpr size_t kBytes = kRing ? (size_t)kStage * kSlots : 0;

    const AddArgs& a;
    const int lane;
    char* const slots;
    int put = 0, get = 0;

    __device__ __forceinline__ Feed(const AddArgs& args, char* smem)
        : a(args), lane(threadIdx.x % TPR), slots(smem) {}

    // A copy of N bytes, 16 or 8, and where a thread's chunk lies that has `before` bytes a thread
    // in front of it.
    template <int N>
    static __device__ __forceinline__ void copy(char* to, const void* from) {
        if constexpr (N == 16)
            ptx::cp_async16(to, from);
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(to)), "l"(from)
                         : "memory");
    }
    template <int N>
    static __device__ __forceinline__ char* slot(char* stage, int before) {
        return stage + before * kThreads + threadIdx.x * N;
    }

    // f(source, type of its chunk, bytes in front) for what a row has
    template <typename F>
    __device__ __forceinline__ void each(int row, F f) {
        const bool with_x = BWD ? a.da != nullptr : a.x != nullptr;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            if (row >= a.T || c >= a.D) continue;
            const long long e = (long long)row * a.D + c;
            int at = i * (kR + kT) * (BWD ? 2 : 1);
            f(static_cast<const R*>(a.r) + row * a.r_stride + c, Chunk<R, E>{}, at);
            at += kR;
            if (with_x) f(static_cast<const T*>(a.x) + row * a.x_stride + c, Chunk<T, E>{}, at);
            at += kT;
            if constexpr (BWD) {
                f(static_cast<const T*>(a.dy) + e, Chunk<T, E>{}, at);
                at += kT;
                if (a.dr) f(static_cast<const R*>(a.dr) + e, Chunk<R, E>{}, at);
            }
        }
    }
    __device__ __forceinline__ void start(int row) {
        if constexpr (kRing) {
            char* to = slots + put * kStage;
            each(row, [&](const void* from, auto chunk, int at) {
                copy<sizeof(chunk)>(slot<sizeof(chunk)>(to, at), from);
            });
            ptx::cp_async_commit();
            put = put + 1 == kSlots ? 0 : put + 1;
        }
    }
    template <typename C>
    __device__ __forceinline__ void take(C& c, int at) {
        c = *reinterpret_cast<const C*>(slot<sizeof(C)>(slots + get * kStage, at));
    }
    // The row whose copies were begun first, zeros where it has nothing.
    __device__ __forceinline__ void finish(int row, Row<R, T, E, NC, BWD>& o) {
        const bool with_x = BWD ? a.da != nullptr : a.x != nullptr;
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            const bool in = row < a.T && c < a.D;
            o.r[i].zero();
            o.x[i].zero();
            if constexpr (BWD) {
                o.y[i].zero();
                o.u[i].zero();
            }
            if (!in) continue;
            if constexpr (kRing) {
                int at = i * (kR + kT) * (BWD ? 2 : 1);
                take(o.r[i], at);
                at += kR;
                if (with_x) take(o.x[i], at);
                at += kT;
                if constexpr (BWD) {
                    take(o.y[i], at);
                    at += kT;
                    if (a.dr) take(o.u[i], at);
                }
            } else {
                const long long e = (long long)row * a.D + c;
                o.r[i].load(static_cast<const R*>(a.r) + row * a.r_stride + c);
                if (with_x) o.x[i].load(static_cast<const T*>(a.x) + row * a.x_stride + c);
                if constexpr (BWD) {
                    o.y[i].load(static_cast<const T*>(a.dy) + e);
                    if (a.dr) o.u[i].load(static_cast<const R*>(a.dr) + e);
                }
            }
        }
        get = get + 1 == kSlots ? 0 : get + 1;
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
__global__ void __launch_bounds__(Rows<TPR>::kThreads, Rows<TPR>::kMin) add_fwd_kernel(const AddArgs a) {
    using F = Feed<R, T, E, TPR, NC, false>;
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    extern __shared__ __align__(16) char slots[];
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    int row = blockIdx.x * RPC + group, turn = 0;
    F feed(a, slots);
#pragma unroll
    for (int k = 0; k < F::kAhead; ++k) feed.start(row + k * step);
    for (; row - group < a.T; row += step, ++turn) {
        Row<R, T, E, NC, false> cur;
        feed.finish(row, cur);
        float v[NC][E];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            cur.r[i].get(v[i]);
            if (a.x) {
                float f[E], al[E];
                cur.x[i].get(f);
                alphas(a, (i * TPR + lane) * E, al);
                vfma(v[i], al, f, v[i]);
            }
            vdot(sum, v[i], v[i]);
        }
        feed.start(row + F::kAhead * step);
        sum.x += sum.y;
        sum = row_sum<TPR, false>(sum, red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            if (row >= a.T || c >= a.D) continue;
            const long long e = (long long)row * a.D + c;
            if (a.r_out) Chunk<R, E>::store(static_cast<R*>(a.r_out) + e, v[i]);
            float w[E];
            a.w.get(c, w);
            vmul(w, w, inv);
            vmul(v[i], v[i], w);
            Chunk<T, E>::store(static_cast<T*>(a.y) + e, v[i]);
        }
    }
}

template <typename R, typename T, int E, int TPR, int NC>
__global__ void __launch_bounds__(Rows<TPR>::kThreads, Rows<TPR>::kMin) add_bwd_kernel(const AddArgs a) {
    using F = Feed<R, T, E, TPR, NC, true>;
    constexpr int RPC = Rows<TPR>::kRows, W = Rows<TPR>::kThreads / 32;
    extern __shared__ __align__(16) char slots[];
    __shared__ float2 red[TPR > 32 ? 2 * W : 1];
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, step = gridDim.x * RPC;
    const float inv_d = 1.f / a.D;
    float dw[NC][E] = {}, da[NC][E] = {};
    int row = blockIdx.x * RPC + group, turn = 0;
    F feed(a, slots);
#pragma unroll
    for (int k = 0; k < F::kAhead; ++k) feed.start(row + k * step);
    for (; row - group < a.T; row += step, ++turn) {
        Row<R, T, E, NC, true> cur;
        feed.finish(row, cur);
        float2 s2 = make_float2(0.f, 0.f), sn = s2;   // sums of r^2 and of dn r
        float dn[NC][E];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            float v[E], y[E], w[E] = {};
            cur.r[i].get(v);
            cur.y[i].get(y);
            if (c < a.D) a.w.get(c, w);
            vmul(dn[i], y, w);
            vdot(s2, v, v);
            vdot(sn, dn[i], v);
        }
        feed.start(row + F::kAhead * step);
        const float2 sum = row_sum<TPR, true>(make_float2(s2.x + s2.y, sn.x + sn.y), red, turn, W);
        const float inv = rsqrtf(fmaf(sum.x, inv_d, a.eps));
        const float m = inv * (inv * (sum.y * inv_d));   // (inv * inv may overflow)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (i * TPR + lane) * E;
            if (row >= a.T || c >= a.D) continue;
            const long long e = (long long)row * a.D + c;
            float v[E], y[E], f[E], d[E];
            cur.r[i].get(v);
            cur.y[i].get(y);
            cur.u[i].get(d);
            cur.x[i].get(f);
            vfma(dn[i], v, -m, dn[i]);
            vfma(d, dn[i], inv, d);                  // dr
            Chunk<R, E>::store(static_cast<R*>(a.dres) + e, d);
            vmul(v, v, inv);
            vfma(dw[i], y, v, dw[i]);
            vfma(da[i], d, f, da[i]);
            if (a.dx) {
                alphas(a, c, f);
                vmul(f, f, d);
                Chunk<T, E>::store(static_cast<T*>(a.dx) + e, f);
            }
        }
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
        constexpr size_t smem = Feed<R, T, E, TPR, NC, false>::kBytes;
        static Resident resident;
        int per_sm = 0;
        if (resident.get(k, N, smem, per_sm) != KDA_OK) return KDA_ERR_CUDA;
        const int grid = grid_of(per_sm, (a.T + RPC - 1) / RPC);
        TimedLaunch tl("add_norm_fwd", s);
        k<<<grid, N, smem, s>>>(a);
        return launch_status();
    }
    static kda_status run(const AddArgs& a, int type, cudaStream_t s) {
        if constexpr (E != 8) {
            if (type == 1) return go<float, float>(a, s);
            if (type == 2) return go<float, __nv_bfloat16>(a, s);
        }
        return go<__nv_bfloat16, __nv_bfloat16>(a, s);
    }
};

template <int E, int TPR, int NC>
struct Bwd {
    template <typename R, typename T>
    static kda_status go(const AddArgs& a, cudaStream_t s) {
        constexpr int N = Rows<TPR>::kThreads, RPC = Rows<TPR>::kRows;
        auto* k = add_bwd_kernel<R, T, E, TPR, NC>;
        constexpr size_t smem = Feed<R, T, E, TPR, NC, true>::kBytes;
        static Resident resident;
        int per_sm = 0;
        if (resident.get(k, N, smem, per_sm) != KDA_OK) return KDA_ERR_CUDA;
        const int grid = std::min(grid_of(per_sm, (a.T + RPC - 1) / RPC), kPartsPerSm * sm_count());
        {
            TimedLaunch tl("add_norm_bwd", s);
            k<<<grid, N, smem, s>>>(a);
        }
        const kda_status st = launch_status();
        if (st != KDA_OK || (!a.dw && !a.da)) return st;
        return sum_parts_launch(a.part, grid, a.D, a.dw, a.da, s);
    }
    static kda_status run(const AddArgs& a, int type, cudaStream_t s) {
        if constexpr (E != 8) {
            if (type == 1) return go<float, float>(a, s);
            if (type == 2) return go<float, __nv_bfloat16>(a, s);
        }
        return go<__nv_bfloat16, __nv_bfloat16>(a, s);
    }
};

// Elements of an access: 8 where all is bf16, else 4, where widths, strides and pointers allow them.
int chunk_of(const AddArgs& a, int type) {
    if (!aligned16({a.r, a.x, a.r_out, a.y, a.dy, a.dr, a.dres, a.dx, a.av.p, a.w.p})) return 1;
    for (int E = type == 0 ? 8 : 4; E >= 4; E /= 2)
        if (a.D % E == 0 && a.r_stride % E == 0 && a.x_stride % E == 0) return E;
    return 1;
}
template <template <int, int, int> class F>
kda_status launch(const AddArgs& a, int type, cudaStream_t s) {
    const int E = chunk_of(a, type);
    if (E == 8) return by_width<F, 8>(a.D, a, type, s);
    return E == 4 ? by_width<F, 4>(a.D, a, type, s) : by_width<F, 1>(a.D, a, type, s);
}

}  // namespace

size_t add_norm_ws_bytes(int T, int D) {
    return align256(2 * (size_t)parts_bound(T) * D * sizeof(float));
}

kda_status add_norm_fwd_launch(const AddArgs& a, int type, cudaStream_t s) {
    return launch<Fwd>(a, type, s);
}

kda_status add_norm_bwd_launch(const AddArgs& a, int type, cudaStream_t s) {
    return launch<Bwd>(a, type, s);
}

}  // namespace kda
