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

#include "kda_block.cuh"
#include "kda_ptx.cuh"
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

// ---- the scan over long sequences ----
//
// A CTA walks along T over a slab of channels, 128 bytes of each token, in tiles of 128 tokens.  A
// lane holds the channels of one 4-byte word (two of bf16, one of float32); each of eight warps
// takes 16 tokens of a tile and scans them from a zero state, keeping for each token its local
// state and the product of the decays up to it.  The warps' maps (A, H) are combined through
// shared memory, and the state that enters a warp's run goes to its tokens by one product each.  So
// the dependent chain of a tile is 16 + 8 steps instead of 128, and the data passes once.
//
// Where slabs are few, a cluster of K CTAs walks along one slab, K tiles at a time: the CTAs'
// maps are combined through distributed shared memory, with one cluster barrier for K tiles.
constexpr int kWarps = 8, kRun = 16, kTile = kWarps * kRun, kThreads = kWarps * 32;
constexpr int kRowBytes = 128, kTileBytes = kTile * kRowBytes;
constexpr int kMaxCluster = 16;

template <typename T>
struct Lane {
    static constexpr int N = 4 / sizeof(T), kSlab = 32 * N;   // channels of a lane, of a slab
    static __device__ __forceinline__ void get(uint32_t w, float (&v)[N]) {
        if constexpr (N == 2)
            unpack2(w, v[0], v[1]);
        else
            v[0] = __uint_as_float(w);
    }
    // all of the lane's channels, or those below C
    static __device__ __forceinline__ void put(T* p, const float (&v)[N], int left, bool word) {
        if constexpr (N == 2) {
            if (word) {
                if (left > 0) *reinterpret_cast<uint32_t*>(p) = pack2(v[0], v[1]);
            } else {
                if (left > 0) p[0] = __float2bfloat16_rn(v[0]);
                if (left > 1) p[1] = __float2bfloat16_rn(v[1]);
            }
        } else {
            if (left > 0) p[0] = v[0];
        }
    }
    static __device__ __forceinline__ void get32(const float* p, float (&v)[N], int left) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = p && left > j ? p[j] : 0.f;
    }
    static __device__ __forceinline__ void put32(float* p, const float (&v)[N], int left) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (left > j) p[j] = v[j];
    }
};

// The map of a run of tokens, h -> A h + H; `cut`: it forgets h.
template <int N>
struct Map {
    float A[N], H[N];
};
template <int N>
__device__ __forceinline__ void apply(const Map<N>& m, bool cut, float (&h)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = cut ? m.H[j] : fmaf(m.A[j], h[j], m.H[j]);
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
// A 16-byte read of another CTA's shared memory, at the address of this one's `p`.
__device__ __forceinline__ float4 read_peer(const void* p, uint32_t rank) {
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ void copy16(void* to, const void* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile of `a` [T][..] at p (channel c0 of token 0) into shared memory, zeros past T and C: a zero
// x, g and do leave states as they are.  WIDE: 16-byte copies in flight; else element by element.
template <typename T, bool WIDE>
__device__ __forceinline__ void fill(char* to, const T* p, long long stride, int t0, int T_, int left) {
    constexpr int E = 16 / sizeof(T);
    if (WIDE) {
#pragma unroll
        for (int i = 0; i < kTileBytes / 16 / kThreads; ++i) {
            const int k = i * kThreads + threadIdx.x, row = k / 8, c = k % 8 * E;
            const bool in = t0 + row < T_ && c < left;
            copy16(to + k * 16, in ? p + (t0 + row) * stride + c : p, in);
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

// The sequences (fewer than 65536) that begin and end at the tokens of a tile.
constexpr unsigned kNone = 0xffff;
struct Marks {
    uint16_t first[kTile], last[kTile];
};
__device__ __forceinline__ void mark(Marks& m, const int* cu, int nseq, int t0, int T) {
    const int i = threadIdx.x, t = t0 + i;
    if (i >= kTile) return;
    unsigned first = kNone, last = kNone;
    if (t < T) {
        int lo = 0, hi = nseq;   // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        if (cu[lo] == t) first = lo;
        if (cu[lo + 1] == t + 1) last = lo;
    }
    m.first[i] = (uint16_t)first;
    m.last[i] = (uint16_t)last;
}

template <int N>
struct __align__(16) Shared {
    float4 map[kWarps][32];          // the warps' maps (A, H); N = 1 uses half of each
    float2 back[kWarps][32];         // backward: H of the map that runs the other way
    float4 mine[2][32];              // this CTA's map, in two turns, read by its cluster
    float4 peers[kMaxCluster][32];   // the cluster's maps
    int cut[kWarps], cut_back[kWarps], mine_cut[2][4], peers_cut[kMaxCluster];
    Marks marks[2];
};

template <int N>
__device__ __forceinline__ float4 to4(const Map<N>& m) {
    return make_float4(m.A[0], m.A[N - 1], m.H[0], m.H[N - 1]);
}
template <int N>
__device__ __forceinline__ Map<N> from4(const float4& v) {
    Map<N> m;
    m.A[0] = v.x;
    m.H[0] = v.z;
    m.A[N - 1] = v.y;
    m.H[N - 1] = v.w;
    return m;
}

// The state that enters this CTA's tile, and behind the cluster's tiles of this turn, from the
// state `carry` before them; tiles in the order of the ranks (or against it).
template <int N, bool BACK>
__device__ __forceinline__ void combine(Shared<N>& sh, int K, int rank, int turn, const Map<N>& own,
                                        bool own_cut, float (&carry)[N], float (&enter)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
        sh.mine[turn][lane] = to4<N>(own);
        if (lane == 0) sh.mine_cut[turn][0] = own_cut;
    }
    cluster_sync();
    for (int r = warp; r < K; r += kWarps) {
        sh.peers[r][lane] = read_peer(&sh.mine[turn][lane], r);
        if (lane == 0) sh.peers_cut[r] = __float_as_int(read_peer(&sh.mine_cut[turn][0], r).x);
    }
    __syncthreads();
    for (int i = 0; i < K; ++i) {
        const int r = BACK ? K - 1 - i : i;
        if (r == rank) {
#pragma unroll
            for (int j = 0; j < N; ++j) enter[j] = carry[j];
        }
        apply<N>(from4<N>(sh.peers[r][lane]), sh.peers_cut[r] != 0, carry);
    }
}

constexpr int kFwdStages = 3, kBwdStages = 2;

// VL: a packed batch.  WIDE: 16-byte copies and 4-byte stores.
template <typename T, bool VL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanArgs a, int K) {
    constexpr int N = Lane<T>::N;
    extern __shared__ __align__(128) char stages[];
    Shared<N>& sh = *reinterpret_cast<Shared<N>*>(stages + kFwdStages * 2 * kTileBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = K > 1 ? (int)cluster_rank() : 0, slab = blockIdx.x / K, b = blockIdx.y;
    const int c0 = slab * Lane<T>::kSlab, c = c0 + lane * N, left = a.C - c;
    const int tiles = (a.T + kTile - 1) / kTile, turns = (tiles + K - 1) / K;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c0;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c0;
    T* o = a.o ? static_cast<T*>(a.o) + (long long)b * a.T * a.C + c : nullptr;
    const int every = (a.T + kStateEvery - 1) / kStateEvery;
    float* states = a.states ? a.states + (long long)b * every * a.C + c : nullptr;
    auto h0_of = [&](int s) { return a.h0 ? a.h0 + (long long)s * a.C + c : nullptr; };

    if (VL) {
        const bool bad = bad_cu(a.cu, a.nseq, a.T);
        if (bad && threadIdx.x == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
        // sequences without tokens (all of them, where cu_seqlens is wrong) end as they begin
        for (int s = rank * kWarps + warp; a.ht && s < a.nseq; s += K * kWarps)
            if (bad || a.cu[s] == a.cu[s + 1]) {
                float v[N];
                Lane<T>::get32(h0_of(s), v, left);
                Lane<T>::put32(a.ht + (long long)s * a.C + c, v, left);
            }
        if (bad) return;   // alike in all CTAs of a cluster
    }
    auto load = [&](int turn) {
        if (turn < turns) {
            char* to = stages + turn % kFwdStages * 2 * kTileBytes;
            const int t0 = (turn * K + rank) * kTile;
            fill<T, WIDE>(to, x, a.x_token, t0, a.T, a.C - c0);
            fill<T, WIDE>(to + kTileBytes, g, a.g_token, t0, a.T, a.C - c0);
        }
        copies_commit();
    };
    load(0);
    load(1);
    float carry[N];
    Lane<T>::get32(VL ? nullptr : h0_of(b), carry, left);

    for (int turn = 0; turn < turns; ++turn) {
        const int t0 = (turn * K + rank) * kTile, tw = t0 + warp * kRun;
        Marks& marks = sh.marks[turn & 1];
        if (VL) mark(marks, a.cu, a.nseq, t0, a.T);
        copies_wait<1>();
        __syncthreads();
        load(turn + 2);
        const uint32_t* xs = reinterpret_cast<const uint32_t*>(
                                 stages + turn % kFwdStages * 2 * kTileBytes) + warp * kRun * 32 + lane;
        const uint32_t* gs = xs + kTileBytes / 4;

        // tokens of the run that begin and end a sequence
        unsigned firsts = 0, lasts = 0;
        if (VL) {
            firsts = __ballot_sync(~0u, marks.first[warp * kRun + lane % kRun] != kNone) & 0xffffu;
            lasts = __ballot_sync(~0u, marks.last[warp * kRun + lane % kRun] != kNone) & 0xffffu;
        }
        // from a zero state: each token's local state and product of decays
        float h[kRun][N], P[kRun][N];
        float hc[N], pc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) hc[j] = 0.f, pc[j] = 1.f;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float xv[N], gv[N];
            Lane<T>::get(xs[i * 32], xv);
            Lane<T>::get(gs[i * 32], gv);
            if (VL && (firsts >> i & 1)) Lane<T>::get32(h0_of(marks.first[warp * kRun + i]), hc, left);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float d = decay<T>(gv[j]);
                hc[j] = advance(d, hc[j], a.tied ? rest(d) * xv[j] : xv[j]);
                pc[j] = advance(d, pc[j], 0.f);
                h[i][j] = hc[j];
                P[i][j] = pc[j];
            }
        }
        Map<N> m;
#pragma unroll
        for (int j = 0; j < N; ++j) m.A[j] = pc[j], m.H[j] = hc[j];
        sh.map[warp][lane] = to4<N>(m);
        if (VL && lane == 0) sh.cut[warp] = firsts != 0;
        __syncthreads();

        float enter[N];
        if (K > 1) {
            // the CTA's map, then the cluster's
            Map<N> own = from4<N>(sh.map[0][lane]);
            bool cut = VL && sh.cut[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const Map<N> next = from4<N>(sh.map[w][lane]);
                const bool c1 = VL && sh.cut[w];
                apply<N>(next, c1, own.H);
#pragma unroll
                for (int j = 0; j < N; ++j) own.A[j] *= next.A[j];
                cut |= c1;
            }
            combine<N, false>(sh, K, rank, turn & 1, own, cut, carry, enter);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) enter[j] = carry[j];
        }
        float into[N];   // the state that enters this warp's run
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) {
#pragma unroll
                for (int j = 0; j < N; ++j) into[j] = enter[j];
            }
            apply<N>(from4<N>(sh.map[w][lane]), VL && sh.cut[w], enter);
        }
        if (K == 1) {
#pragma unroll
            for (int j = 0; j < N; ++j) carry[j] = enter[j];
        }

        if (states && tw % kStateEvery == 0 && tw < a.T) {
            float v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = into[j];
            if (VL && (firsts & 1)) Lane<T>::get32(h0_of(marks.first[warp * kRun]), v, left);
            Lane<T>::put32(states + (long long)(tw / kStateEvery) * a.C, v, left);
        }
        const int from = VL && firsts ? __ffs(firsts) - 1 : kRun;   // what entered ends there
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = VL && i >= from ? h[i][j] : fmaf(P[i][j], into[j], h[i][j]);
            if (o && tw + i < a.T) Lane<T>::put(o + (long long)(tw + i) * a.C, v, left, WIDE);
            if (VL && (lasts >> i & 1) && a.ht)
                Lane<T>::put32(a.ht + (long long)marks.last[warp * kRun + i] * a.C + c, v, left);
        }
    }
    if (!VL && a.ht && rank == 0 && warp == 0) Lane<T>::put32(a.ht + (long long)b * a.C + c, carry, left);
    copies_wait<0>();
    if (K > 1) cluster_sync();   // no CTA leaves while another may read its shared memory
}

// Tiles from the last to the first.  The states inside a tile are formed again from the kept ones
// (one each 64 tokens, in 32 bits), so nothing is read of the rounded outputs; the same passes
// carry m the other way.
template <typename T, bool VL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanArgs a, int K) {
    constexpr int N = Lane<T>::N;
    extern __shared__ __align__(128) char stages[];
    Shared<N>& sh = *reinterpret_cast<Shared<N>*>(stages + kBwdStages * 3 * kTileBytes);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = K > 1 ? (int)cluster_rank() : 0, slab = blockIdx.x / K, b = blockIdx.y;
    const int c0 = slab * Lane<T>::kSlab, c = c0 + lane * N, left = a.C - c;
    const int tiles = (a.T + kTile - 1) / kTile, turns = (tiles + K - 1) / K;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + c0;
    const T* g = static_cast<const T*>(a.g) + b * a.g_batch + c0;
    const long long row0 = (long long)b * a.T * a.C;
    const T* dout = static_cast<const T*>(a.dout) + row0 + c0;
    T *dx = static_cast<T*>(a.dx) + row0 + c, *dg = static_cast<T*>(a.dg) + row0 + c;
    const int every = (a.T + kStateEvery - 1) / kStateEvery;
    const float* states = a.states + (long long)b * every * a.C + c;
    auto h0_of = [&](int s) { return a.h0 ? a.h0 + (long long)s * a.C + c : nullptr; };
    auto dht_of = [&](int s) { return a.dht ? a.dht + (long long)s * a.C + c : nullptr; };

    if (VL) {
        const bool bad = bad_cu(a.cu, a.nseq, a.T);
        if (bad && threadIdx.x == 0) atomicCAS(&g_scan_error, 0, (int)KDA_ERR_SHAPE);
        for (int s = rank * kWarps + warp; a.dh0 && s < a.nseq; s += K * kWarps)
            if (bad || a.cu[s] == a.cu[s + 1]) {
                float v[N];
                Lane<T>::get32(dht_of(s), v, left);
                Lane<T>::put32(a.dh0 + (long long)s * a.C + c, v, left);
            }
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
        copies_commit();
    };
    load(0);
    float carry[N];
    Lane<T>::get32(VL ? nullptr : dht_of(b), carry, left);

    for (int turn = 0; turn < turns; ++turn) {
        const int t0 = tile_of(turn) * kTile, tw = t0 + warp * kRun;
        Marks& marks = sh.marks[turn & 1];
        if (VL) mark(marks, a.cu, a.nseq, t0, a.T);
        // the kept state of this warp's 64 tokens
        float into[N];
        const int block = tw / kStateEvery;
        Lane<T>::get32(block < every ? states + (long long)block * a.C : nullptr, into, left);
        copies_wait<0>();
        __syncthreads();
        load(turn + 1);
        const uint32_t* xs = reinterpret_cast<const uint32_t*>(
                                 stages + turn % kBwdStages * 3 * kTileBytes) + warp * kRun * 32 + lane;
        const uint32_t *gs = xs + kTileBytes / 4, *ds = gs + kTileBytes / 4;
        unsigned firsts = 0, lasts = 0;
        if (VL) {
            firsts = __ballot_sync(~0u, marks.first[warp * kRun + lane % kRun] != kNone) & 0xffffu;
            lasts = __ballot_sync(~0u, marks.last[warp * kRun + lane % kRun] != kNone) & 0xffffu;
        }
        // the run's map, and its map the other way (of m), which has the same product of decays
        float d[kRun][N];
        Map<N> m;
        float back[N];
#pragma unroll
        for (int j = 0; j < N; ++j) m.A[j] = 1.f, m.H[j] = 0.f, back[j] = 0.f;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float xv[N], gv[N];
            Lane<T>::get(xs[i * 32], xv);
            Lane<T>::get(gs[i * 32], gv);
            if (VL && (firsts >> i & 1)) Lane<T>::get32(h0_of(marks.first[warp * kRun + i]), m.H, left);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                d[i][j] = decay<T>(gv[j]);
                m.H[j] = advance(d[i][j], m.H[j], a.tied ? rest(d[i][j]) * xv[j] : xv[j]);
                m.A[j] = advance(d[i][j], m.A[j], 0.f);
            }
        }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            float dv[N];
            Lane<T>::get(ds[i * 32], dv);
            if (VL && (lasts >> i & 1)) Lane<T>::get32(dht_of(marks.last[warp * kRun + i]), back, left);
#pragma unroll
            for (int j = 0; j < N; ++j) back[j] = advance(d[i][j], dv[j] + back[j], 0.f);
        }
        sh.map[warp][lane] = to4<N>(m);
        sh.back[warp][lane] = make_float2(back[0], back[N - 1]);
        if (VL && lane == 0) {
            sh.cut[warp] = firsts != 0;
            sh.cut_back[warp] = lasts != 0;
        }
        __syncthreads();

        // the states: from the kept one over the warps before this one
        constexpr int kPer = kStateEvery / kRun;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w / kPer == warp / kPer && w < warp) apply<N>(from4<N>(sh.map[w][lane]), VL && sh.cut[w], into);
        // m: from the end over the warps behind
        auto back_of = [&](int w) {
            Map<N> v = from4<N>(sh.map[w][lane]);
            const float2 e = sh.back[w][lane];
            v.H[0] = e.x;
            v.H[N - 1] = N == 2 ? e.y : e.x;
            return v;
        };
        float enter[N], mc[N];
        if (K > 1) {
            Map<N> own = back_of(kWarps - 1);
            bool cut = VL && sh.cut_back[kWarps - 1];
#pragma unroll
            for (int w = kWarps - 2; w >= 0; --w) {
                const Map<N> next = back_of(w);
                const bool c1 = VL && sh.cut_back[w];
                apply<N>(next, c1, own.H);
#pragma unroll
                for (int j = 0; j < N; ++j) own.A[j] *= next.A[j];
                cut |= c1;
            }
            combine<N, true>(sh, K, rank, turn & 1, own, cut, carry, enter);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) enter[j] = carry[j];
        }
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
            if (w == warp) {
#pragma unroll
                for (int j = 0; j < N; ++j) mc[j] = enter[j];
            }
            apply<N>(back_of(w), VL && sh.cut_back[w], enter);
        }
        if (K == 1) {
#pragma unroll
            for (int j = 0; j < N; ++j) carry[j] = enter[j];
        }

        float before[kRun][N];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float xv[N];
            Lane<T>::get(xs[i * 32], xv);
            if (VL && (firsts >> i & 1)) Lane<T>::get32(h0_of(marks.first[warp * kRun + i]), into, left);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                before[i][j] = a.tied ? into[j] - xv[j] : into[j];
                into[j] = advance(d[i][j], into[j], a.tied ? rest(d[i][j]) * xv[j] : xv[j]);
            }
        }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            float dv[N], dxv[N], dgv[N];
            Lane<T>::get(ds[i * 32], dv);
            if (VL && (lasts >> i & 1)) Lane<T>::get32(dht_of(marks.last[warp * kRun + i]), mc, left);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float l = dv[j] + mc[j];
                mc[j] = advance(d[i][j], l, 0.f);
                dxv[j] = a.tied ? rest(d[i][j]) * l : l;
                dgv[j] = mc[j] * before[i][j];
            }
            if (tw + i < a.T) {
                Lane<T>::put(dx + (long long)(tw + i) * a.C, dxv, left, WIDE);
                Lane<T>::put(dg + (long long)(tw + i) * a.C, dgv, left, WIDE);
            }
            if (VL && (firsts >> i & 1) && a.dh0)
                Lane<T>::put32(a.dh0 + (long long)marks.first[warp * kRun + i] * a.C + c, mc, left);
        }
    }
    if (!VL && a.dh0 && rank == 0 && warp == 0) Lane<T>::put32(a.dh0 + (long long)b * a.C + c, carry, left);
    copies_wait<0>();
    if (K > 1) cluster_sync();
}

// CTAs of a cluster: as many as keep all slabs' CTAs resident (two per SM), tiles allowing.
int cluster_of(long long slabs, int T) {
    int K = 1;
    while (K < kMaxCluster && 2 * K * slabs <= 2 * sm_count() && K * kTile < T) K *= 2;
    return K;
}

template <typename T, bool BWD, bool VL, bool WIDE>
kda_status launch(const ScanArgs& a, cudaStream_t s) {
    auto* k = BWD ? scan_bwd_kernel<T, VL, WIDE> : scan_fwd_kernel<T, VL, WIDE>;
    const int slabs = (a.C + Lane<T>::kSlab - 1) / Lane<T>::kSlab;
    const int K = cluster_of((long long)slabs * a.B, a.T);
    const size_t smem = (BWD ? kBwdStages * 3 : kFwdStages * 2) * kTileBytes + sizeof(Shared<Lane<T>::N>);
    // once per device; a second time does no harm
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
            cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return KDA_ERR_CUDA;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
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
    return cudaLaunchKernelEx(&cfg, k, a, K) == cudaSuccess ? launch_status() : KDA_ERR_CUDA;
}

template <typename T, bool BWD>
kda_status pick(const ScanArgs& a, cudaStream_t s) {
    constexpr int E = 16 / sizeof(T);
    const bool wide = a.C % E == 0 && a.x_batch % E == 0 && a.x_token % E == 0 && a.g_batch % E == 0 &&
                      a.g_token % E == 0 && aligned16({a.x, a.g, a.o, a.dout, a.dx, a.dg});
    if (a.cu) return wide ? launch<T, BWD, true, true>(a, s) : launch<T, BWD, true, false>(a, s);
    return wide ? launch<T, BWD, false, true>(a, s) : launch<T, BWD, false, false>(a, s);
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
    return bf16 ? pick<__nv_bfloat16, false>(a, s) : pick<float, false>(a, s);
}

kda_status scan_bwd_launch(const ScanArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? pick<__nv_bfloat16, true>(a, s) : pick<float, true>(a, s);
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
