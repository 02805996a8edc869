// The gated linear recurrence, per channel:
//
//     h_t = exp(g_t) h_{t-1} + c_t x_t,  c_t = 1, or 1 - exp(g_t) (tied),  o_t = h_t
//     m_t = exp(g_t) l_t,  l_t = do_t + m_{t+1}      (m behind the last token: dht)
//     dx_t = c_t l_t,  dg_t = m_t (h_{t-1} - [tied] x_t),  dh0 = m_1
//
// Each step is an affine map of the state, so runs of tokens combine: a run is (A, H) with
// A = prod exp(g), H its end state from zero, and maps h to A h + H.  A packed batch is one line
// of tokens with a map that forgets what came before at every first token.
#include <atomic>
#include <mutex>
#include <type_traits>

#include "kda_block.cuh"
#include "kda_exchange.cuh"
#include "kda_ptx.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_scan_error = 0;   // a kda_status

namespace {

using namespace block;

constexpr int kStateEvery = KDA_SCAN_STATE_EVERY;   // tokens between kept states

// A lane's channels, and packed arithmetic on the two of bf16.
template <int N>
struct V {
    float v[N];
};
__device__ __forceinline__ V<1> fma(V<1> a, V<1> b, V<1> c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
__device__ __forceinline__ V<1> mul(V<1> a, V<1> b) { return {{a.v[0] * b.v[0]}}; }
__device__ __forceinline__ V<1> add(V<1> a, V<1> b) { return {{a.v[0] + b.v[0]}}; }
__device__ __forceinline__ float2 f2(V<2> a) { return make_float2(a.v[0], a.v[1]); }
__device__ __forceinline__ V<2> v2(float2 a) { return {{a.x, a.y}}; }
__device__ __forceinline__ V<2> fma(V<2> a, V<2> b, V<2> c) { return v2(__ffma2_rn(f2(a), f2(b), f2(c))); }
__device__ __forceinline__ V<2> mul(V<2> a, V<2> b) { return v2(__fmul2_rn(f2(a), f2(b))); }
__device__ __forceinline__ V<2> add(V<2> a, V<2> b) { return v2(__fadd2_rn(f2(a), f2(b))); }
template <int N>
__device__ __forceinline__ V<N> all(float x) {
    V<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = x;
    return r;
}

// The decay exp(g) as keep + d, keep = 1 or 0, held in d alone.  For g in (-1/4, -0] keep is 1 and
// d = exp(g) - 1 <= -0: a rounded exp(g) close to one would be off by that rounding in each of the
// thousands of tokens that it acts over.  Else keep is 0 and d = exp(g) > 0: h + (exp(g) - 1) h would
// lose what is small beside h.  exp(g) - 1 is the Taylor series of six terms, its next one under
// 2^-24 there; exp(g), by the fast power of two (2^-22 of it, and the rounding of its argument), has
// 2^-126 added to it, so that d stays above 0 where it underflows.  (As integers, the bits of the
// numbers from -0 down to -1/4 are the least of all.)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int N>
__device__ __forceinline__ V<N> decay(V<N> g, V<N>& keep) {
    V<N> p = fma(g, all<N>(1.f / 720.f), all<N>(1.f / 120.f));
    p = fma(g, p, all<N>(1.f / 24.f));
    p = fma(g, p, all<N>(1.f / 6.f));
    p = fma(g, p, all<N>(1.f / 2.f));
    p = fma(g, p, all<N>(1.f));
    p = mul(g, p);
    V<N> e = mul(g, all<N>(1.44269504f));
#pragma unroll
    for (int j = 0; j < N; ++j) e.v[j] = exp2_fast(e.v[j]);
    e = add(e, all<N>(1.17549435e-38f));
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const bool near = __float_as_int(g.v[j]) < __float_as_int(-0.25f);
        p.v[j] = near ? p.v[j] : e.v[j];
        keep.v[j] = near ? 1.f : 0.f;
    }
    return p;
}
// keep, from d's sign
template <int N>
__device__ __forceinline__ V<N> kept(V<N> d) {
    V<N> k;
#pragma unroll
    for (int j = 0; j < N; ++j) k.v[j] = __int_as_float(__float_as_int(d.v[j]) >> 31 & 0x3f800000);
    return k;
}
// The same, formed again and not taken from an earlier pass: held since then it would need
// registers that are not there.
template <int N>
__device__ __forceinline__ V<N> kept_again(V<N> d) {
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+f"(d.v[j]));
    return kept(d);
}
// exp(g) h, and with an input
template <int N>
__device__ __forceinline__ V<N> decayed(V<N> d, V<N> k, V<N> h) {
    return fma(k, h, mul(d, h));
}
template <int N>
__device__ __forceinline__ V<N> advance(V<N> d, V<N> k, V<N> h, V<N> u) {
    return fma(k, h, fma(d, h, u));
}
template <int N>
__device__ __forceinline__ V<N> less(V<N> a, V<N> b) {
    V<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = a.v[j] - b.v[j];
    return r;
}
// (1 - exp(g)) x; 1 - keep is exact
template <int N>
__device__ __forceinline__ V<N> remainder(V<N> d, V<N> k, V<N> x) {
    V<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = (1.f - k.v[j]) - d.v[j];
    return mul(r, x);
}

// ---- the scan over long sequences ----
//
// A CTA walks along T over a slab of channels, 128 bytes of each token, in tiles of 128 tokens.  A
// lane holds the channels of one 4-byte word (two of bf16, one of float32); each of eight warps
// takes 16 tokens of a tile and scans them from a zero state, keeping for each token its local
// state and the product of the decays up to it.  The warps' maps (A, H) are combined through
// shared memory, and the state that enters a warp's run goes to its tokens by one product each.  So
// the dependent chain of a tile is 16 + 8 steps instead of 128, and the data passes once.
//
// Where slabs are few, a cluster of K CTAs walks along one slab, K tiles at a time.  Each CTA
// pushes its tile's map into the others' shared memory (asynchronous stores that complete on the
// receiver's mbarrier: a cluster barrier would wait for the outputs' stores each time).
//
// What bounds it: 3 elements a step forward and 5 backward are the floor, but a turn of tiles takes
// 1.3 us forward and 2.3 backward with one CTA to an SM, 2.2 to 2.6 and 4.1 with two: the chain scan,
// barrier, combine, barrier, and 21, 36 and (tied) 46 instructions an element at half of the
// issue slots.  With 256 CTAs busy that is near HBM, with fewer it is not.  One GB300, in a graph:
//   4 x 8192 x 2048 bf16      forward 82 us, 4.95 TB/s (0.74); backward 129 us, 5.2 TB/s (0.78), tied 152 us
//   1 x 65536 x 512 float32   forward, tied 87 us, 4.6 TB/s (0.69; 16 slabs, clusters of 13)
//   1 x 65536 x 512 bf16      forward 82 us, 2.5 TB/s (0.37; 8 slabs, clusters of 12); backward 123 us
//   1 x 65536 x 1024 float32  forward, tied 132 us, 6.1 TB/s (0.91; 32 slabs, clusters of 8)
//   32768 x 1000 bf16 in 16 packed sequences, tied, forward 98 us (0.30), backward 156 us, 2.1 TB/s (0.32)
// (The hot loops are at 128 registers, and a condition more or less around the exchange moves these times by
// 2 to 10 %: the compiler then spills, or orders the loops in another way.)
// A thread per channel, token by token: 4.7 ms and 7.4 ms for the first, 48 ms for the second.
constexpr int kWarps = 8, kRun = 16, kTile = kWarps * kRun, kThreads = kWarps * 32;
constexpr int kRowBytes = 128, kTileBytes = kTile * kRowBytes;
constexpr int kMaxCluster = 16;
constexpr long long kWaitCycles = 4000000000ll;   // about two seconds

template <typename T>
struct Lane {
    static constexpr int N = 4 / sizeof(T), kSlab = 32 * N;   // channels of a lane, of a slab
    static __device__ __forceinline__ V<N> get(uint32_t w) {
        V<N> r;
        if constexpr (N == 2)
            unpack2(w, r.v[0], r.v[1]);
        else
            r.v[0] = __uint_as_float(w);
        return r;
    }
    // two values: a token's two channels, or one channel of two tokens
    static __device__ __forceinline__ V<2> pair(const uint32_t* w) {
        if constexpr (N == 2)
            return get(w[0]);
        else
            return {{__uint_as_float(w[0]), __uint_as_float(w[32])}};
    }
    // the lane's channels (`left` of them are inside C), in one word or each by itself
    template <bool WORD>
    static __device__ __forceinline__ void put(T* p, const V<N>& r, int left) {
        if constexpr (N == 2) {
            if (WORD) {
                if (left > 0) *reinterpret_cast<uint32_t*>(p) = pack2(r.v[0], r.v[1]);
            } else {
                if (left > 0) p[0] = __float2bfloat16_rn(r.v[0]);
                if (left > 1) p[1] = __float2bfloat16_rn(r.v[1]);
            }
        } else {
            if (left > 0) p[0] = r.v[0];
        }
    }
    static __device__ __forceinline__ V<N> get32(const float* p, int left) {
        V<N> r;
#pragma unroll
        for (int j = 0; j < N; ++j) r.v[j] = p && left > j ? p[j] : 0.f;
        return r;
    }
    static __device__ __forceinline__ void put32(float* p, const V<N>& r, int left) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (left > j) p[j] = r.v[j];
    }
};

// token i's channels of such a pair
template <int N>
__device__ __forceinline__ V<N> part(const V<2>& p, int i) {
    V<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = p.v[N == 2 ? j : i];
    return r;
}

// The map of a run of tokens, h -> A h + H.  In a packed batch a run in which a sequence begins
// forgets h: its A is then a NaN with bits that no arithmetic makes.
constexpr uint32_t kCut = 0x7fc0c0deu;
template <int N>
struct Map {
    V<N> A, H;
};
template <int N>
__device__ __forceinline__ bool is_cut(const Map<N>& m) {
    return __float_as_uint(m.A.v[0]) == kCut;
}
template <bool VL, int N>
__device__ __forceinline__ V<N> apply(const Map<N>& m, V<N> h) {
    const V<N> r = fma(m.A, h, m.H);
    return VL && is_cut(m) ? m.H : r;
}
// first, then next
template <bool VL, int N>
__device__ __forceinline__ Map<N> compose(const Map<N>& first, const Map<N>& next) {
    Map<N> r;
    r.H = apply<VL>(next, first.H);
    r.A = mul(first.A, next.A);
    if (VL && (is_cut(first) || is_cut(next))) r.A = all<N>(__uint_as_float(kCut));
    return r;
}
template <int N>
__device__ __forceinline__ float4 to4(const Map<N>& m) {
    return make_float4(m.A.v[0], m.A.v[N - 1], m.H.v[0], m.H.v[N - 1]);
}
template <int N>
__device__ __forceinline__ Map<N> from4(const float4& v) {
    Map<N> m;
    m.A.v[0] = v.x;
    m.H.v[0] = v.z;
    m.A.v[N - 1] = v.y;
    m.H.v[N - 1] = v.w;
    return m;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    return at;
}
// 16 bytes into a peer's shared memory; they count on its mbarrier.
__device__ __forceinline__ void push16(uint32_t to, uint32_t bar, const float4& v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::
                     "r"(to), "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
                 "r"(__float_as_uint(v.w)), "r"(bar)
                 : "memory");
}
// A wait that gives up, and says so, after `limit` cycles.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, long long limit) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (clock64() - t0 > limit) {
            atomicExch(&g_scan_error, (int)KDA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void prefetch(const void* p) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}
__device__ __forceinline__ void copy16(void* to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile of `a` [T][..] at p (channel c0 of token 0) into shared memory, zeros past T and C: a zero
// x, g and do leave states as they are.  WIDE: 16-byte copies in flight; else element by element.
template <typename T, bool WIDE>
__device__ __forceinline__ void fill(char* to, const T* p, long long stride, int t0, int T_, int left) {
    constexpr int E = 16 / sizeof(T), kCopies = kTileBytes / 16 / kThreads;
    if (WIDE) {
        const int row0 = threadIdx.x / 8, c = threadIdx.x % 8 * E;
        const T* from = p + (t0 + row0) * stride + c;
        to += threadIdx.x * 16;
        if (t0 + kTile <= T_ && left >= Lane<T>::kSlab) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i, from += kThreads / 8 * stride)
                ptx::cp_async16(to + i * kThreads * 16, from);
        } else {
            const int rows = c < left ? T_ - t0 - row0 : 0;
#pragma unroll
            for (int i = 0; i < kCopies; ++i, from += kThreads / 8 * stride) {
                const bool in = i * (kThreads / 8) < rows;
                copy16(to + i * kThreads * 16, in ? from : p, in);
            }
        }
    } else {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 4
        for (int i = 0; i < kRun; ++i) {
            const int row = i * kWarps + warp;
#pragma unroll
            for (int j = 0; j < Lane<T>::N; ++j) {
                const int c = lane + 32 * j;
                T v = from_f<T>(0.f);
                if (t0 + row < T_ && c < left) v = p[(t0 + row) * stride + c];
                reinterpret_cast<T*>(to)[row * Lane<T>::kSlab + c] = v;
            }
        }
    }
}

// cu_seqlens must rise from 0 to T.
__device__ bool bad_cu(const int* cu, int nseq, int T) {
    bool bad = cu[0] != 0 || cu[nseq] != T;
    for (int i = threadIdx.x; i < nseq; i += blockDim.x) bad |= cu[i] < 0 || cu[i] > cu[i + 1];
    return __syncthreads_or(bad);
}

// The tokens of a warp's run that begin and end a sequence, as bits, and these sequences, for token
// i in lane i.  A run inside the sequence that was last looked up needs no look-up.
struct Marks {
    unsigned firsts = 0, lasts = 0;
    int first = 0, last = 0;
    int begin = 0, end = 0;   // of that sequence

    template <bool BACK>
    __device__ __forceinline__ void look_up(const int* cu, int nseq, int tw, int T) {
        firsts = lasts = 0;
        if (tw > begin && tw + kRun < end) return;
        const int t = tw + (threadIdx.x & 31) % kRun;
        bool begins = false, ends = false;
        int from = 0, to = 0;
        if (t < T) {
            int lo = 0, hi = nseq;   // cu[lo] <= t < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            first = last = lo;
            from = cu[lo];
            to = cu[lo + 1];
            begins = from == t;
            ends = to == t + 1;
        }
        firsts = __ballot_sync(~0u, begins) & ((1u << kRun) - 1);
        lasts = __ballot_sync(~0u, ends) & ((1u << kRun) - 1);
        begin = __shfl_sync(~0u, from, BACK ? 0 : kRun - 1);
        end = __shfl_sync(~0u, to, BACK ? 0 : kRun - 1);
    }
    __device__ __forceinline__ bool any() const { return (firsts | lasts) != 0; }
};

struct __align__(16) Shared {
    float4 peers[2][kMaxCluster][32];   // maps of the cluster's CTAs, in two turns
    uint64_t arrived[2];                // ... and that they are here
    int lost[32];                       // the turns in which lanes' waits gave up
};

// Exchanges of a cluster's maps, one a turn, by one warp of each CTA, as kda_exchange.cuh tells them.
struct Exchange {
    Shared& sh;
    const int K, rank, turns;
    long long limit = kWaitCycles;
    static constexpr unsigned kMapBytes = 32 * sizeof(float4);

    // Before the first turn; also a barrier of the cluster.
    __device__ __forceinline__ void begin(bool clear) {
        if (clear && threadIdx.x < 32) sh.lost[threadIdx.x] = -1;
        if (threadIdx.x == 0) {
            for (int i = 0; i < 2; ++i) ptx::mbar_init(&sh.arrived[i], 1);
            ptx::fence_mbar_init();
            for (int i = 0; i < 2; ++i) ptx::mbar_arrive_expect_tx(&sh.arrived[i], K * kMapBytes);
        }
        cluster_sync();
    }
    // A lane's wait of a turn; that it gave up is kept.
    __device__ __forceinline__ bool wait_of(int turn) {
        if (await(&sh.arrived[turn & 1], turn >> 1 & 1, limit)) return true;
        sh.lost[threadIdx.x & 31] = turn;
        return false;
    }
    __device__ __forceinline__ int lost_turn(int lane) const {
        return *static_cast<volatile const int*>(&sh.lost[lane]);
    }

    // What exchange_drain asks for.
    __device__ __forceinline__ bool wait(int turn) {
        return await(&sh.arrived[turn & 1], turn >> 1 & 1, limit);
    }
    __device__ __forceinline__ void expect(int turn, int n) {
        ptx::mbar_expect_tx(&sh.arrived[turn & 1], n * K * kMapBytes);
    }
    __device__ __forceinline__ void arrive(int turn) { ptx::mbar_arrive(&sh.arrived[turn & 1]); }
    __device__ __forceinline__ void pause() {
        for (const long long t0 = clock64(); clock64() - t0 < limit;) {}
    }
};

template <bool VL, int N, bool BACK>
struct Cluster : Exchange {
    // Whether this lane's wait gave up is held in a register, backward in shared memory alone.  (There the
    // register makes 176 us of 156 in a packed pass; forward the reads make 88 of 82.)
    static constexpr bool kLostInMemory = BACK;
    bool lost = false;

    __device__ __forceinline__ void begin() { Exchange::begin(kLostInMemory); }
    // After the last turn; also a barrier of the cluster.  A CTA may end then: nothing comes to its shared
    // memory any more.
    __device__ __forceinline__ void end() {
        cluster_sync();
        const bool gone = kLostInMemory ? threadIdx.x == 0 && lost_turn(0) >= 0 : lost && (threadIdx.x & 31) == 0;
        if (gone) exchange_drain(*static_cast<Exchange*>(this), K, turns, sh.lost[0]);
    }

    // The state that enters this CTA's tile; `carry` goes from before the cluster's tiles of this
    // turn to behind them.  Tiles in the order of the ranks, or against it.
    __device__ __forceinline__ V<N> exchange(int turn, const Map<N>& own, V<N>& carry) {
        const int lane = threadIdx.x & 31, i = turn & 1;
#pragma unroll 4
        for (int r = 0; r < K; ++r)
            push16(peer_address(&sh.peers[i][rank][lane], r), peer_address(&sh.arrived[i], r), to4<N>(own));
        bool gone = kLostInMemory ? lost_turn(lane) >= 0 : lost;
        if (!gone && !wait_of(turn)) gone = true;
        lost = gone;
        __syncwarp();
        if (lane == 0 && !gone) ptx::mbar_arrive_expect_tx(&sh.arrived[i], K * kMapBytes);
        const int step = BACK ? -1 : 1;
        int r = BACK ? K - 1 : 0;
#pragma unroll 4
        for (; r != rank; r += step) carry = apply<VL>(from4<N>(sh.peers[i][r][lane]), carry);
        const V<N> enter = carry;
#pragma unroll 4
        for (; r != (BACK ? -1 : K); r += step) carry = apply<VL>(from4<N>(sh.peers[i][r][lane]), carry);
        return enter;
    }

    // What enters each warp's run, from the warps' maps: map_of(w)[0], in the order of the warps or
    // against it, left at into_of(w).
    template <typename M, typename I>
    __device__ __forceinline__ void enter_runs(int turn, V<N>& carry, M map_of, I into_of) {
        Map<N> m[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m[w] = from4<N>(*map_of(BACK ? kWarps - 1 - w : w));
        V<N> into = carry;
        if (K > 1) {
            Map<N> sum = m[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) sum = compose<VL>(sum, m[w]);
            into = exchange(turn, sum, carry);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            *into_of(BACK ? kWarps - 1 - w : w) = make_float2(into.v[0], into.v[N - 1]);
            into = apply<VL>(m[w], into);
        }
        if (K == 1) carry = into;
    }
};
template <int N>
__device__ __forceinline__ V<N> from2(const float2& v) {
    V<N> r;
    r.v[0] = v.x;
    r.v[N - 1] = N == 2 ? v.y : v.x;
    return r;
}

// Keeps the compiler from moving the loads of an unrolled pass to its beginning, where they would
// take registers that are not there.
__device__ __forceinline__ void hold_loads() { asm volatile("" ::: "memory"); }

constexpr int kFwdStages = 3, kBwdStages = 2;

// VL: a packed batch.  WIDE: 16-byte copies and 4-byte stores.
template <typename T, bool TIED, bool VL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanArgs a, int K) {
    constexpr int N = Lane<T>::N, S = 2 / N;   // tokens of a pair of values
    extern __shared__ __align__(128) char stages[];
    Shared& sh = *reinterpret_cast<Shared*>(stages + kFwdStages * 2 * kTileBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = K > 1 ? (int)cluster_rank() : 0, slab = blockIdx.x / K, b = blockIdx.y;
    const int c0 = slab * Lane<T>::kSlab, c = c0 + lane * N, left = a.C - c;
    const int tiles = (a.T + kTile - 1) / kTile, turns = (tiles + K - 1) / K;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c0;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c0;
    const int every = (a.T + kStateEvery - 1) / kStateEvery;
    float* states = a.states ? a.states + (long long)b * every * a.C + c : nullptr;
    auto h0_of = [&](int s) { return a.h0 ? a.h0 + (long long)s * a.C + c : nullptr; };

    if (VL) {
        const bool bad = bad_cu(a.cu, a.nseq, a.T);
        if (bad && threadIdx.x == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
        // sequences without tokens (all of them, where cu_seqlens is wrong) end as they begin
        for (int s = rank * kWarps + warp; a.ht && s < a.nseq; s += K * kWarps)
            if (bad || a.cu[s] == a.cu[s + 1])
                Lane<T>::put32(a.ht + (long long)s * a.C + c, Lane<T>::get32(h0_of(s), left), left);
        if (bad) return;   // alike in all CTAs of a cluster
    }
    auto load = [&](int turn) {
        if (turn < turns) {
            char* to = stages + turn % kFwdStages * 2 * kTileBytes;
            const int t0 = (turn * K + rank) * kTile;
            fill<T, WIDE>(to, x, a.x_token, t0, a.T, a.C - c0);
            fill<T, WIDE>(to + kTileBytes, g, a.g_token, t0, a.T, a.C - c0);
        }
        ptx::cp_async_commit();
    };
    load(0);
    load(1);
    // one warp combines the maps; not the same one in CTAs that share an SM
    const int lead = blockIdx.x % kWarps;
    Cluster<VL, N, false> cluster{{sh, K, rank, turns}};
    if (K > 1) cluster.begin();
    V<N> carry = Lane<T>::get32(VL ? nullptr : h0_of(b), left);
    Marks marks;

    for (int turn = 0; turn < turns; ++turn) {
        const int t0 = (turn * K + rank) * kTile, tw = t0 + warp * kRun;
        if (VL) marks.look_up<false>(a.cu, a.nseq, tw, a.T);
        // runs with a border in them take code of their own: its tests at each token would keep the
        // tokens of the others apart, too
        const bool marked = VL && marks.any();
        auto first_state = [&](int i) {
            return Lane<T>::get32(h0_of(__shfl_sync(~0u, marks.first, i)), left);
        };
        auto last_state = [&](int i, V<N> v) {
            const int s = __shfl_sync(~0u, marks.last, i);
            if (a.ht) Lane<T>::put32(a.ht + (long long)s * a.C + c, v, left);
        };
        if (VL && a.h0 && marks.firsts) {   // (shuffles need the whole warp, lanes past C too)
            const int s = __shfl_sync(~0u, marks.first, __ffs(marks.firsts) - 1);
            if (left > 0) prefetch(h0_of(s));
        }
        copies_wait<1>();
        __syncthreads();
        load(turn + 2);
        char* stage = stages + turn % kFwdStages * 2 * kTileBytes;
        const uint32_t* xs = reinterpret_cast<uint32_t*>(stage) + warp * kRun * 32 + lane;
        const uint32_t* gs = xs + kTileBytes / 4;
        // the warps' maps go where their rows of g were, and what enters their runs behind them
        auto map_of = [&](int w) {
            return reinterpret_cast<float4*>(stage + kTileBytes + w * kRun * kRowBytes) + lane;
        };
        auto into_of = [&](int w) { return reinterpret_cast<float2*>(map_of(w) - lane + 32) + lane; };

        // from a zero state: each token's local state and product of decays
        V<N> h[kRun], P[kRun];
        Map<N> m = {all<N>(1.f), all<N>(0.f)};
        auto scan = [&](auto with_marks) {
            constexpr bool M = decltype(with_marks)::value;
#pragma unroll
            for (int p = 0; p < kRun; p += S) {
                V<2> k2, u2 = Lane<T>::pair(xs + p * 32);
                const V<2> d2 = decay(Lane<T>::pair(gs + p * 32), k2);
                if (TIED) u2 = remainder(d2, k2, u2);
#pragma unroll
                for (int i = p; i < p + S; ++i) {
                    const V<N> d = part<N>(d2, i - p), k = part<N>(k2, i - p), u = part<N>(u2, i - p);
                    if (M) {
                        P[i] = d;   // (the tests below would keep these, too, in order)
                        h[i] = u;
                    } else {
                        m.H = advance(d, k, m.H, u);
                        m.A = decayed(d, k, m.A);
                        h[i] = m.H;
                        P[i] = m.A;
                    }
                }
            }
            if constexpr (M) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    if (marks.firsts >> i & 1) {   // what enters the run ends here
                        m.H = first_state(i);
                        m.A = all<N>(0.f);
                    }
                    const V<N> k = kept(P[i]);
                    m.H = advance(P[i], k, m.H, h[i]);
                    m.A = decayed(P[i], k, m.A);
                    h[i] = m.H;
                    P[i] = m.A;
                }
            }
        };
        if (marked)
            scan(std::true_type{});
        else
            scan(std::false_type{});
        if (VL && marks.firsts) m.A = all<N>(__uint_as_float(kCut));
        __syncwarp();
        *map_of(warp) = to4<N>(m);
        __syncthreads();

        if (warp == lead) cluster.enter_runs(turn, carry, map_of, into_of);
        __syncthreads();
        V<N> into = from2<N>(*into_of(warp));

        if (states && tw % kStateEvery == 0 && tw < a.T) {
            const V<N> v = VL && (marks.firsts & 1) ? first_state(0) : into;
            Lane<T>::put32(states + (long long)(tw / kStateEvery) * a.C, v, left);
        }
        const int rows = a.o ? a.T - tw : 0;   // alike in all lanes: what follows shuffles
        T* o = static_cast<T*>(a.o) + ((long long)b * a.T + tw) * a.C + c;
        auto write = [&](auto with_marks, auto whole) {
            constexpr bool M = decltype(with_marks)::value, W = decltype(whole)::value;
#pragma unroll
            for (int i = 0; i < kRun; ++i, o += a.C) {
                if (M && (marks.firsts >> i & 1)) into = all<N>(0.f);
                const V<N> v = fma(P[i], into, h[i]);
                if (W || i < rows) Lane<T>::template put<WIDE>(o, v, left);
                if (M && (marks.lasts >> i & 1)) last_state(i, v);
            }
        };
        if (marked)
            write(std::true_type{}, std::false_type{});
        else if (rows >= kRun)
            write(std::false_type{}, std::true_type{});
        else
            write(std::false_type{}, std::false_type{});
    }
    if (!VL && a.ht && rank == 0 && warp == lead) Lane<T>::put32(a.ht + (long long)b * a.C + c, carry, left);
    copies_wait<0>();
    if (K > 1) cluster.end();
}

// Tiles from the last to the first.  The states inside a tile are formed again from the kept ones
// (one each 64 tokens, in 32 bits), so nothing is read of the rounded outputs; the same passes
// carry m the other way.
template <typename T, bool TIED, bool VL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanArgs a, int K) {
    constexpr int N = Lane<T>::N, S = 2 / N;   // tokens of a pair of values
    extern __shared__ __align__(128) char stages[];
    Shared& sh = *reinterpret_cast<Shared*>(stages + kBwdStages * 3 * kTileBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = K > 1 ? (int)cluster_rank() : 0, slab = blockIdx.x / K, b = blockIdx.y;
    const int c0 = slab * Lane<T>::kSlab, c = c0 + lane * N, left = a.C - c;
    const int tiles = (a.T + kTile - 1) / kTile, turns = (tiles + K - 1) / K;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c0;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c0;
    const T* dout = static_cast<const T*>(a.dout) + (long long)b * a.T * a.C + c0;
    const int every = (a.T + kStateEvery - 1) / kStateEvery;
    const float* states = a.states + (long long)b * every * a.C + c;
    auto h0_of = [&](int s) { return a.h0 ? a.h0 + (long long)s * a.C + c : nullptr; };
    auto dht_of = [&](int s) { return a.dht ? a.dht + (long long)s * a.C + c : nullptr; };

    if (VL) {
        const bool bad = bad_cu(a.cu, a.nseq, a.T);
        if (bad && threadIdx.x == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
        for (int s = rank * kWarps + warp; a.dh0 && s < a.nseq; s += K * kWarps)
            if (bad || a.cu[s] == a.cu[s + 1])
                Lane<T>::put32(a.dh0 + (long long)s * a.C + c, Lane<T>::get32(dht_of(s), left), left);
        if (bad) return;
    }
    // tile of a turn: the cluster's tiles from behind
    auto tile_of = [&](int turn) { return (turns - 1 - turn) * K + rank; };
    auto load = [&](int turn) {
        if (turn < turns) {
            char* to = stages + turn % kBwdStages * 3 * kTileBytes;
            const int t0 = tile_of(turn) * kTile;
            fill<T, WIDE>(to, x, a.x_token, t0, a.T, a.C - c0);
            fill<T, WIDE>(to + kTileBytes, g, a.g_token, t0, a.T, a.C - c0);
            fill<T, WIDE>(to + 2 * kTileBytes, dout, a.C, t0, a.T, a.C - c0);
        }
        ptx::cp_async_commit();
    };
    load(0);
    // one warp combines the maps of m, one those of the states
    constexpr int kPer = kStateEvery / kRun;
    const int lead = blockIdx.x % kWarps, second = (lead + 2) % kWarps;
    Cluster<VL, N, true> cluster{{sh, K, rank, turns}};
    if (K > 1) cluster.begin();
    V<N> carry = Lane<T>::get32(VL ? nullptr : dht_of(b), left);
    Marks marks;

    for (int turn = 0; turn < turns; ++turn) {
        const int t0 = tile_of(turn) * kTile, tw = t0 + warp * kRun;
        if (VL) marks.look_up<true>(a.cu, a.nseq, tw, a.T);
        // runs with a border in them take code of their own: its tests at each token would keep the
        // tokens of the others apart, too
        const bool marked = VL && marks.any();
        auto first_state = [&](int i) {
            return Lane<T>::get32(h0_of(__shfl_sync(~0u, marks.first, i)), left);
        };
        auto last_grad = [&](int i) {
            return Lane<T>::get32(dht_of(__shfl_sync(~0u, marks.last, i)), left);
        };
        auto first_grad = [&](int i, V<N> v) {
            const int s = __shfl_sync(~0u, marks.first, i);
            if (a.dh0) Lane<T>::put32(a.dh0 + (long long)s * a.C + c, v, left);
        };
        if (VL && a.h0 && marks.firsts) {   // (shuffles need the whole warp, lanes past C too)
            const int s = __shfl_sync(~0u, marks.first, __ffs(marks.firsts) - 1);
            if (left > 0) prefetch(h0_of(s));
        }
        if (VL && a.dht && marks.lasts) {
            const int s = __shfl_sync(~0u, marks.last, 31 - __clz(marks.lasts));
            if (left > 0) prefetch(dht_of(s));
        }
        V<N> into, kept_state[kWarps / kPer];
        if (warp == second) {
#pragma unroll
            for (int i = 0; i < kWarps / kPer; ++i) {
                const int block = t0 / kStateEvery + i;
                kept_state[i] = Lane<T>::get32(block < every ? states + (long long)block * a.C : nullptr, left);
            }
        }
        copies_wait<0>();
        __syncthreads();
        load(turn + 1);
        char* stage = stages + turn % kBwdStages * 3 * kTileBytes;
        const uint32_t* xs = reinterpret_cast<uint32_t*>(stage) + warp * kRun * 32 + lane;
        const uint32_t *gs = xs + kTileBytes / 4, *ds = gs + kTileBytes / 4;
        // the warps' maps go where their rows of g were: that of m and that of the states, and behind
        // them what enters their runs
        auto back_of = [&](int w) {
            return reinterpret_cast<float4*>(stage + kTileBytes + w * kRun * kRowBytes) + lane;
        };
        auto map_of = [&](int w) { return back_of(w) + 32; };
        auto m_of = [&](int w) { return reinterpret_cast<float2*>(back_of(w) - lane + 64) + lane; };
        auto into_of = [&](int w) { return m_of(w) + 32; };
        V<N> d[kRun];
        Map<N> m = {all<N>(1.f), all<N>(0.f)}, back = m;
        auto scan = [&](auto with_marks) {
            constexpr bool M = decltype(with_marks)::value;
#pragma unroll
            for (int p = 0; p < kRun; p += S) {
                V<2> k2, u2 = Lane<T>::pair(xs + p * 32);
                const V<2> d2 = decay(Lane<T>::pair(gs + p * 32), k2);
                if (TIED) u2 = remainder(d2, k2, u2);
#pragma unroll
                for (int i = p; i < p + S; ++i) {
                    d[i] = part<N>(d2, i - p);
                    const V<N> k = part<N>(k2, i - p);
                    if (M) continue;   // (the tests below would keep the decays, too, in order)
                    m.H = advance(d[i], k, m.H, part<N>(u2, i - p));
                    m.A = decayed(d[i], k, m.A);
                }
            }
            if constexpr (M) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    const V<N> k = kept(d[i]), xv = Lane<T>::get(xs[i * 32]);
                    if (marks.firsts >> i & 1) m.H = first_state(i);
                    m.H = advance(d[i], k, m.H, TIED ? remainder(d[i], k, xv) : xv);
                    m.A = decayed(d[i], k, m.A);
                }
            }
            back.A = m.A;
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i) {
                if (M && (marks.lasts >> i & 1)) back.H = last_grad(i);
                back.H = decayed(d[i], kept(d[i]), add(Lane<T>::get(ds[i * 32]), back.H));
            }
        };
        if (marked)
            scan(std::true_type{});
        else
            scan(std::false_type{});
        if (VL && marks.firsts) m.A = all<N>(__uint_as_float(kCut));
        if (VL && marks.lasts) back.A = all<N>(__uint_as_float(kCut));
        __syncwarp();
        *map_of(warp) = to4<N>(m);
        *back_of(warp) = to4<N>(back);
        __syncthreads();

        if (warp == lead) cluster.enter_runs(turn, carry, back_of, m_of);
        if (warp == second) {
            // the states that enter the runs, from those kept each kPer runs
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w % kPer == 0) into = kept_state[w / kPer];
                *into_of(w) = make_float2(into.v[0], into.v[N - 1]);
                into = apply<VL>(from4<N>(*map_of(w)), into);
            }
        }
        __syncthreads();
        into = from2<N>(*into_of(warp));
        V<N> mc = from2<N>(*m_of(warp));

        const int rows = a.T - tw;   // alike in all lanes: what follows shuffles
        const long long end = ((long long)b * a.T + tw + kRun - 1) * a.C + c;
        T *dx = static_cast<T*>(a.dx) + end, *dg = static_cast<T*>(a.dg) + end;
        // h_{t-1}, less x where tied.  Tied with two channels to a lane these do not fit into the
        // registers (spilled, at 10 % of L1 hits, they took 237 us for 163): they go where this
        // run's x and g were.  (8 bytes of other values are still spilled.)
        constexpr bool kStash = TIED && N == 2;
        V<N> w[kStash ? 1 : kRun];
        uint32_t *stash = const_cast<uint32_t*>(xs), *stash2 = const_cast<uint32_t*>(gs);
        auto keep_w = [&](int i, const V<N>& v) {
            if constexpr (kStash) {
                stash[i * 32] = __float_as_uint(v.v[0]);
                stash2[i * 32] = __float_as_uint(v.v[N - 1]);
            } else {
                w[i] = v;
            }
        };
        auto w_of = [&](int i) {
            if constexpr (kStash) {
                V<N> v;
                v.v[0] = __uint_as_float(stash[i * 32]);
                v.v[N - 1] = __uint_as_float(stash2[i * 32]);
                return v;
            } else {
                return w[i];
            }
        };
        if (kStash) __syncwarp();   // what entered the run, among g's rows, has been read
        auto write = [&](auto with_marks, auto whole) {
            constexpr bool M = decltype(with_marks)::value, W = decltype(whole)::value;
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (i % 4 == 0) hold_loads();
                const V<N> xv = Lane<T>::get(xs[i * 32]), k = TIED ? kept_again(d[i]) : kept(d[i]);
                if (M && (marks.firsts >> i & 1)) into = first_state(i);
                keep_w(i, TIED ? less(into, xv) : into);
                into = advance(d[i], k, into, TIED ? remainder(d[i], k, xv) : xv);
            }
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i, dx -= a.C, dg -= a.C) {
                if (i % 4 == 3) hold_loads();
                if (M && (marks.lasts >> i & 1)) mc = last_grad(i);
                const V<N> k = TIED ? kept_again(d[i]) : kept(d[i]), l = add(Lane<T>::get(ds[i * 32]), mc);
                mc = decayed(d[i], k, l);
                if (W || i < rows) {
                    Lane<T>::template put<WIDE>(dx, TIED ? remainder(d[i], k, l) : l, left);
                    Lane<T>::template put<WIDE>(dg, mul(mc, w_of(i)), left);
                }
                if (M && (marks.firsts >> i & 1)) first_grad(i, mc);
            }
        };
        if (marked)
            write(std::true_type{}, std::false_type{});
        else if (rows >= kRun)
            write(std::false_type{}, std::true_type{});
        else
            write(std::false_type{}, std::false_type{});
    }
    if (!VL && a.dh0 && rank == 0 && warp == lead) Lane<T>::put32(a.dh0 + (long long)b * a.C + c, carry, left);
    copies_wait<0>();
    if (K > 1) cluster.end();
}

// What a kernel needs once per device: its attributes, and how many clusters of each size the
// device holds at once (sizes of nine to sixteen fit badly into its parts: 14 clusters of 16 CTAs,
// where 36 of 8 fit).
struct Setup {
    std::atomic<bool> ready{false};
    std::mutex lock;
    int clusters[kMaxCluster + 1];
    int alone[kMaxCluster + 1];   // with one CTA to an SM
};
template <typename K>
bool prepare(Setup& s, K kernel, size_t smem) {
    if (s.ready.load(std::memory_order_acquire)) return true;
    std::lock_guard<std::mutex> hold(s.lock);
    if (s.ready.load(std::memory_order_relaxed)) return true;
    constexpr size_t kAloneBytes = 120 * 1024;   // two of these do not fit an SM
    static_assert(kAloneBytes >= (kBwdStages * 3) * kTileBytes + sizeof(Shared), "");
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAloneBytes) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();   // said here, not by the next call
        return false;
    }
    auto count = [&](int k, size_t bytes) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)k, 1, 1};
        cfg.gridDim = dim3(k);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = bytes;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
        cudaGetLastError();
        return 0;
    };
    for (int k = 1; k <= kMaxCluster; ++k) {
        s.clusters[k] = count(k, smem);
        s.alone[k] = count(k, kAloneBytes);   // (asked about, never launched)
    }
    s.ready.store(true, std::memory_order_release);
    return true;
}
// CTAs of a cluster: the size with the least time for its turns one after the other, over all the
// rounds that the slabs need.  A turn takes about 1.75 times as long where CTAs share an SM (forward
// 1.3 us alone and 2.2 to 2.6 shared, backward 2.3 and 4.1), which they do not where the device has
// room for all of them one to an SM.  (Times by size, the chosen last: 16 slabs of 65536 float32 tokens 124 us
// with 6, 139 with 7, 90 with 13; 8 slabs of bf16 104 us with 16, 82 with 12; 160 slabs of 8192 tokens 138 us with
// 1, 110 with 5.  One factor for both directions: 4 x 8192 x 2048 bf16 forward takes 79 us with 1 and 82 with 2,
// backward 144 and 129.)
int cluster_of(const Setup& s, long long slabs, int T) {
    const int tiles = (T + kTile - 1) / kTile;
    long long best = -1;
    int K = 1;
    for (int k = 1; k <= kMaxCluster && k <= tiles; ++k) {
        if (s.clusters[k] < 1) continue;
        const long long turns = (slabs + s.clusters[k] - 1) / s.clusters[k] * ((tiles + k - 1) / k);
        const long long cost = turns * (slabs <= s.alone[k] ? 4 : 7);
        if (best < 0 || cost < best) {
            best = cost;
            K = k;
        }
    }
    return K;
}

template <typename T, bool BWD, bool TIED, bool VL, bool WIDE>
kda_status launch(const ScanArgs& a, cudaStream_t s) {
    auto* k = BWD ? scan_bwd_kernel<T, TIED, VL, WIDE> : scan_fwd_kernel<T, TIED, VL, WIDE>;
    const int slabs = (a.C + Lane<T>::kSlab - 1) / Lane<T>::kSlab;
    const size_t smem = (BWD ? kBwdStages * 3 : kFwdStages * 2) * kTileBytes + sizeof(Shared);
    static Setup setups[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || !prepare(setups[dev], k, smem))
        return KDA_ERR_CUDA;
    const int K = cluster_of(setups[dev], (long long)slabs * a.B, a.T);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(slabs * K, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)K, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    TimedLaunch tl(BWD ? "gated_scan_bwd" : "gated_scan_fwd", s);
    cudaLaunchKernelEx(&cfg, k, a, K);
    return launch_status();
}

template <typename T, bool BWD, bool TIED>
kda_status pick(const ScanArgs& a, cudaStream_t s) {
    constexpr int E = 16 / sizeof(T);
    const bool wide = a.C % E == 0 && a.x_batch % E == 0 && a.x_token % E == 0 && a.g_batch % E == 0 &&
                      a.g_token % E == 0 && aligned16({a.x, a.g, a.o, a.dout, a.dx, a.dg});
    if (a.cu) return wide ? launch<T, BWD, TIED, true, true>(a, s) : launch<T, BWD, TIED, true, false>(a, s);
    return wide ? launch<T, BWD, TIED, false, true>(a, s) : launch<T, BWD, TIED, false, false>(a, s);
}

// Diagnostic: the exchange by itself, one warp to a CTA, maps h -> h + (turn + 1) (rank + 1).  CTA
// slow_cta waits `stall` cycles before slow_turn.
__global__ void __launch_bounds__(32) exchange_kernel(int K, int turns, int slow_cta, int slow_turn,
                                                      long long stall, long long limit, float* sums) {
    __shared__ Shared sh;
    const int rank = (int)cluster_rank();
    Cluster<false, 1, false> cluster{{sh, K, rank, turns, limit}};
    cluster.begin();
    V<1> carry = all<1>(0.f);
    for (int turn = 0; turn < turns; ++turn) {
        if (rank == slow_cta && turn == slow_turn)
            for (const long long t0 = clock64(); clock64() - t0 < stall;) {}
        __syncwarp();
        cluster.exchange(turn, {all<1>(1.f), all<1>((float)((turn + 1) * (rank + 1)))}, carry);
    }
    cluster.end();
    if (threadIdx.x == 0) sums[rank] = cluster.lost ? -1.f : carry.v[0];
}

// One token per row, the state read and written once: 256 x 2048 bf16 2.4 us, a launch's time.
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
            V<1> k;
            const V<1> d = decay(V<1>{{gv[j]}}, k), v = {{xv[j]}};
            h[j] = advance(d, k, V<1>{{h[j]}}, tied ? remainder(d, k, v) : v).v[0];
        }
        Chunk<float, E>::store(next + b * C + c, h);
        Chunk<T, E>::store(o + b * C + c, h);
    }
}

template <typename T>
kda_status step(int B, int C, bool tied, const void* x, long long x_row, const void* g,
                long long g_row, const float* state, float* next, void* o, cudaStream_t s) {
    TimedLaunch tl("gated_scan_step", s);
    const bool wide = C % 4 == 0 && x_row % 4 == 0 && g_row % 4 == 0 &&
                      aligned16({x, g, state, next, o});
    const long long n = (long long)B * (wide ? C / 4 : C);
    const int grid = (int)std::min<long long>((n + 255) / 256, 8ll * sm_count());
    auto* k = wide ? step_kernel<T, 4> : step_kernel<T, 1>;
    k<<<grid, 256, 0, s>>>(B, C, tied, static_cast<const T*>(x), x_row, static_cast<const T*>(g), g_row,
                           state, next, static_cast<T*>(o));
    return launch_status();
}

}  // namespace

kda_status scan_fwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s) {
    if (a.tied) return bf16 ? pick<__nv_bfloat16, false, true>(a, s) : pick<float, false, true>(a, s);
    return bf16 ? pick<__nv_bfloat16, false, false>(a, s) : pick<float, false, false>(a, s);
}

kda_status scan_bwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s) {
    if (a.tied) return bf16 ? pick<__nv_bfloat16, true, true>(a, s) : pick<float, true, true>(a, s);
    return bf16 ? pick<__nv_bfloat16, true, false>(a, s) : pick<float, true, false>(a, s);
}

kda_status scan_step_launch(int B, int C, bool bf16, bool tied, const void* x, long long x_row,
                            const void* g, long long g_row, const float* state, float* next,
                            void* o, cudaStream_t s) {
    return bf16 ? step<__nv_bfloat16>(B, C, tied, x, x_row, g, g_row, state, next, o, s)
                : step<float>(B, C, tied, x, x_row, g, g_row, state, next, o, s);
}

kda_status scan_selftest_exchange(int K, int turns, int slow_cta, int slow_turn, long long stall,
                                  long long limit, float* sums, cudaStream_t s) {
    if (cudaFuncSetAttribute(exchange_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return KDA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(K);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)K, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, exchange_kernel, K, turns, slow_cta, slow_turn, stall, limit, sums);
    return launch_status();
}

int* scan_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_scan_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace kda
