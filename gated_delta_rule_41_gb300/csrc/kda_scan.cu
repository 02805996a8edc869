// The gated linear recurrence, per channel:
//
//     h_t = exp(g_t) h_{t-1} + c_t x_t,  c_t = 1, or 1 - exp(g_t) (tied),  o_t = h_t
//     m_t = exp(g_t) l_t,  l_t = do_t + m_{t+1}      (m behind the last token: dht)
//     dx_t = c_t l_t,  dg_t = m_t (h_{t-1} - [tied] x_t),  dh0 = m_1
//
// Each step is an affine map of the state, so runs of tokens combine: a run is (A, H) with
// A = prod exp(g), H its end state from zero, and maps h to A h + H.  A packed batch is one line
// of tokens with a map that forgets what came before at every first token.
#include "kda_block.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_scan_error = 0;   // a kda_status

namespace {

using namespace block;

constexpr int kStateEvery = KDA_SCAN_STATE_EVERY;   // tokens between kept states

// The decay exp(g) as keep + d, keep = 1 or 0, held in d alone: d = exp(g) - 1 <= 0 (keep = 1) for
// g in (-1/4, 0], since a rounded exp(g) close to one would be off by that rounding in each of the
// thousands of tokens that it acts over; else d = exp(g) > 0 (keep = 0), since h + (exp(g) - 1) h
// would lose what is small beside h.  exp(g) - 1 is the Taylor series of six terms, its next one
// under 2^-24 there.  A decay that underflows counts as 2^-126.
template <typename T>
__device__ __forceinline__ float decay(float g) {
    float p = fmaf(g, 1.f / 6.f, 1.f);
    p = fmaf(g * (1.f / 5.f), p, 1.f);
    p = fmaf(g * (1.f / 4.f), p, 1.f);
    p = fmaf(g * (1.f / 3.f), p, 1.f);
    p = fmaf(g * (1.f / 2.f), p, 1.f);
    float e = sizeof(T) == 2 ? __expf(g) : expf(g);
    e = e < 1.17549435e-38f ? 1.17549435e-38f : e;
    return g > -0.25f && g <= 0.f ? g * p : e;
}
__device__ __forceinline__ float kept(float d) { return d > 0.f ? 0.f : 1.f; }
// exp(g) h + u
__device__ __forceinline__ float advance(float d, float h, float u) {
    return fmaf(kept(d), h, fmaf(d, h, u));
}
// 1 - exp(g)
__device__ __forceinline__ float rest(float d) { return (1.f - kept(d)) - d; }

// cu_seqlens must rise from 0 to T.
__device__ bool bad_cu(const int* cu, int nseq, int T) {
    bool bad = cu[0] != 0 || cu[nseq] != T;
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) bad |= cu[i] < 0 || cu[i] > cu[i + 1];
    return __syncthreads_or(bad);
}

// A thread per channel, tokens one after the other.
template <typename T>
__global__ void scan_fwd_kernel(const ScanArgs a) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    const bool bad = a.cu && bad_cu(a.cu, a.nseq, a.T);
    if (bad && c == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
    if (c >= a.C) return;
    const int n = a.cu ? a.nseq : 1, every = (a.T + kStateEvery - 1) / kStateEvery;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c;
    for (int s = 0; s < n; ++s) {
        const int row = a.cu ? s : b, from = a.cu && !bad ? a.cu[s] : 0;
        const int to = bad ? 0 : a.cu ? a.cu[s + 1] : a.T;
        float h = a.h0 ? a.h0[(long long)row * a.C + c] : 0.f;
        for (int t = from; t < to; ++t) {
            if (a.states && t % kStateEvery == 0)
                a.states[((long long)b * every + t / kStateEvery) * a.C + c] = h;
            const float d = decay<T>(to_f<T>(g[t * a.g_token])), v = to_f<T>(x[t * a.x_token]);
            h = advance(d, h, a.tied ? rest(d) * v : v);
            if (a.o) static_cast<T*>(a.o)[((long long)b * a.T + t) * a.C + c] = from_f<T>(h);
        }
        if (a.ht) a.ht[(long long)row * a.C + c] = h;
    }
}

template <typename T>
__global__ void scan_bwd_kernel(const ScanArgs a) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    const bool bad = a.cu && bad_cu(a.cu, a.nseq, a.T);
    if (bad && c == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
    if (c >= a.C) return;
    const int n = a.cu ? a.nseq : 1, every = (a.T + kStateEvery - 1) / kStateEvery;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c;
    for (int s = 0; s < n; ++s) {
        const int row = a.cu ? s : b, from = a.cu && !bad ? a.cu[s] : 0;
        const int to = bad ? 0 : a.cu ? a.cu[s + 1] : a.T;
        float m = a.dht ? a.dht[(long long)row * a.C + c] : 0.f;
        for (int hi = to; hi > from;) {
            const int lo = max(from, (hi - 1) / kStateEvery * kStateEvery);
            float before[kStateEvery];
            float h = lo % kStateEvery == 0
                          ? a.states[((long long)b * every + lo / kStateEvery) * a.C + c]
                          : a.h0 ? a.h0[(long long)row * a.C + c] : 0.f;
            for (int t = lo; t < hi; ++t) {
                before[t - lo] = h;
                const float d = decay<T>(to_f<T>(g[t * a.g_token])), v = to_f<T>(x[t * a.x_token]);
                h = advance(d, h, a.tied ? rest(d) * v : v);
            }
            for (int t = hi - 1; t >= lo; --t) {
                const long long at = ((long long)b * a.T + t) * a.C + c;
                const float d = decay<T>(to_f<T>(g[t * a.g_token])), v = to_f<T>(x[t * a.x_token]);
                const float l = to_f<T>(static_cast<const T*>(a.dout)[at]) + m;
                m = advance(d, l, 0.f);
                static_cast<T*>(a.dx)[at] = from_f<T>(a.tied ? rest(d) * l : l);
                static_cast<T*>(a.dg)[at] = from_f<T>(m * (a.tied ? before[t - lo] - v : before[t - lo]));
            }
            hi = lo;
        }
        if (a.dh0) a.dh0[(long long)row * a.C + c] = m;
    }
}

// One token per row, the state read and written once.
template <typename T, int E>
__global__ void __launch_bounds__(256) step_kernel(int B, int C, bool tied, const T* x, long long x_row,
                                                   const T* g, long long g_row, const float* state,
                                                   float* next, T* o) {
    const long long per = C / E, n = B * per;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const long long b = i / per;
        const int c = (int)(i - b * per) * E;
        Chunk<T, E> xr, gr;
        Chunk<float, E> hr;
        xr.load(x + b * x_row + c);
        gr.load(g + b * g_row + c);
        hr.load(state + b * C + c);
        float xv[E], gv[E], h[E];
        xr.get(xv);
        gr.get(gv);
        hr.get(h);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float d = decay<T>(gv[j]);
            h[j] = advance(d, h[j], tied ? rest(d) * xv[j] : xv[j]);
        }
        Chunk<float, E>::store(next + b * C + c, h);
        Chunk<T, E>::store(o + b * C + c, h);
    }
}

template <typename T>
kda_status step(int B, int C, bool tied, const void* x, long long x_row, const void* g,
                long long g_row, const float* state, float* next, void* o, cudaStream_t s) {
    TimedLaunch tl("gated_scan_step", s);
    const bool wide = C % 8 == 0 && x_row % 8 == 0 && g_row % 8 == 0 &&
                      aligned16({x, g, state, next, o});
    const long long n = (long long)B * (wide ? C / 8 : C);
    const int grid = (int)std::min<long long>((n + 255) / 256, 8ll * sm_count());
    auto* k = wide ? step_kernel<T, 8> : step_kernel<T, 1>;
    k<<<grid, 256, 0, s>>>(B, C, tied, static_cast<const T*>(x), x_row, static_cast<const T*>(g), g_row,
                           state, next, static_cast<T*>(o));
    return launch_status();
}

}  // namespace

kda_status scan_fwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s) {
    TimedLaunch tl("gated_scan_fwd", s);
    const dim3 grid((a.C + 63) / 64, a.B);
    if (bf16)
        scan_fwd_kernel<__nv_bfloat16><<<grid, 64, 0, s>>>(a);
    else
        scan_fwd_kernel<float><<<grid, 64, 0, s>>>(a);
    return launch_status();
}

kda_status scan_bwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s) {
    TimedLaunch tl("gated_scan_bwd", s);
    const dim3 grid((a.C + 63) / 64, a.B);
    if (bf16)
        scan_bwd_kernel<__nv_bfloat16><<<grid, 64, 0, s>>>(a);
    else
        scan_bwd_kernel<float><<<grid, 64, 0, s>>>(a);
    return launch_status();
}

kda_status scan_step_launch(int B, int C, bool bf16, bool tied, const void* x, long long x_row,
                            const void* g, long long g_row, const float* state, float* next,
                            void* o, cudaStream_t s) {
    return bf16 ? step<__nv_bfloat16>(B, C, tied, x, x_row, g, g_row, state, next, o, s)
                : step<float>(B, C, tied, x, x_row, g, g_row, state, next, o, s);
}

int* scan_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_scan_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace kda
