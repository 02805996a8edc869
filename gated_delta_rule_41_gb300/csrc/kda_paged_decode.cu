// Attention of one new token per sequence over a paged key-value cache.
//
// For a key head and its G query heads the work is one pass over the visible
// rows of K and V: 4 G flop for each element read, so HBM bounds it (G = 4,
// bf16: 8 flop a byte) as long as the products run on the tensor cores.  The
// plan is therefore about keeping loads in flight and all SMs equally busy:
//
// * Work is cut into tiles (16 tokens for each warp) of one (sequence, key head,
//   block of query heads).  The tiles of all of them form one line, of which each
//   resident CTA takes an equal stretch (a prefix sum over the lengths, taken
//   by every CTA for itself), so a few long rows spread over the SMs like many
//   unequal ones.  The end of a row counts for three tiles: it costs the CTA
//   as much (counted for none, a batch with many short rows took 56 us against 40).
// * A warp owns 16 tokens of a tile at a time.  They lie in one page (pages are
//   multiples of 16), so one table entry, read a step ahead, gives their
//   addresses.  K and V come by 16-byte asynchronous copies into the warp's own
//   ring of stages, which runs on over the ends of rows: while a row is
//   finished, the copies of the next one are on their way.  Rows that the
//   query does not see are filled with zeros instead of being read.
// * At the end of a row its other warps leave their sums in shared memory, in the
//   order of the MMA fragments, and go on; the first adds them to its own.  A row
//   that lies in one stretch is written at once; of the others each CTA leaves
//   its part, and the CTA that arrives last joins the parts, always in the same
//   order, so the result does not depend on which one that is.
// * S^T = K Q^T has the tokens on the M axis of mma.m16n8k16 and 8 query heads
//   on N, O^T = V^T P the channels on M, so up to 8 heads cost 16 MMAs for 16
//   tokens.  The transposed weights come from movmatrix.
// * Softmax: a running maximum m per head and warp, raised (and the sums
//   rescaled) only when a logit exceeds it by more than 2^8 in weight; the sums
//   are fp32.  Beside e4m3 codes, which are exact in fp16, the weights enter the
//   product with V in fp16 (2^-11), with 2^7 at the maximum, so that only weights
//   below 2^-21 of it leave the normal range (and are rounded by up to 2^-32 of
//   it); beside bf16 values in two bf16 terms (2^-16), since one alone (2^-8)
//   would cost as much as the output's own rounding and the second product is
//   free here.
//
// * K and V rows of 128 bytes or less (D = 64, or e4m3) of two neighbouring heads
//   are taken by one CTA side by side, two warps each: HBM gives pieces of 128
//   bytes at 0.87 of the rate of longer ones (128 window rows of 64 channels: 39 us
//   with one head per CTA, 36 with two, 38 with four, whose parts take longer to join).
//
// Measured: a call costs about 9 us beside its bytes (5 to start and find its
// work, 3 to join rows that several CTAs share), which then pass at the copy
// rate (64 rows of 2048 tokens 49 us, of 4096 89 us: 6.8 TB/s between them).
// 64 rows of 200 to 8192 tokens, 16 heads over 4, D = 128, bf16: 51 us in a graph, 5.5
// TB/s, and DRAM reads 283.2 MB, what the rows hold.  Two CTAs on an SM with D = 128,
// three with D = 64 (the window rows: 46 us against 40 then); more make no
// difference, and neither do smaller shares handed out as CTAs get done.
#include "kda_paged.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_paged_decode_error = 0;   // a kda_status

namespace {

using namespace paged;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGroup = 16;                 // tokens of a warp's step
constexpr int kRowEnd = 3;                 // tiles that the end of a row counts for
// log2 of the weight at the running maximum (weights reach 2^8 times that)
template <bool E4M3>
constexpr float kLow = E4M3 ? 7.f : 0.f;

__device__ __forceinline__ void record() {
    atomicCAS(&g_paged_decode_error, 0, (int)KDA_ERR_SHAPE);
}

// The visible tokens of a query as groups of 16: those of the sinks, then
// those from the window's start on.
struct Span {
    int len, low, sinks;     // token j is seen iff j < len and (j >= low or j < sinks)
    int nsink, first, n;     // groups of sinks; first group of the window; groups in all
    __device__ __forceinline__ int group(int i) const { return i < nsink ? i : i - nsink + first; }
    // tiles of TW warps; a row's length in the line of tiles: its end costs time too
    template <int TW>
    __device__ __forceinline__ int tiles() const {
        return max(1, (n + TW - 1) / TW);
    }
    template <int TW>
    __device__ __forceinline__ int slots() const {
        return tiles<TW>() + kRowEnd;
    }
};
__device__ __forceinline__ Span make_span(const PagedArgs& a, int len) {
    Span s;
    s.len = len;
    s.low = a.window ? max(0, len - a.window) : 0;
    s.sinks = min(a.sinks, s.low);
    s.first = s.low / kGroup;
    s.nsink = min((s.sinks + kGroup - 1) / kGroup, s.first);
    s.n = s.nsink + (len + kGroup - 1) / kGroup - s.first;
    return s;
}
__device__ __forceinline__ int seq_len(const PagedArgs& a, int s) {
    const int len = a.lens[s];
    if (len >= 0 && len <= a.cap) return len;
    record();
    return 0;
}

template <int D, bool E4M3, int NH>
struct Shape {
    static constexpr int RB = D * (E4M3 ? 1 : 2);        // bytes of a row
    static constexpr int RC = RB / 16;                   // 16-byte chunks of a row
    static constexpr int TILE = kGroup * RB;             // K (or V) of a step
    // CTAs of an SM, and the stages of a warp's ring (as many as fit)
    static constexpr int OCC = NH == 2 || D == 128 ? 2 : 3;
    static constexpr int STAGES = RB == 256   ? (NH == 1 ? 3 : 2)
                                  : RB == 128 ? (OCC == 3 ? 4 : D == 64 || NH == 1 ? 6 : 5)
                                              : 8;
    static constexpr int RING = STAGES * 2 * TILE;       // bytes per warp
    static constexpr int KS = D / 16;                    // k steps of S, m tiles of O
    // what a warp knows of a row, per lane: O fragments, maxima, sums
    static constexpr int FRAG = KS * NH + NH;            // float4
    static constexpr size_t SMEM = kWarps * RING + (kWarps - 1) * FRAG * 512;
    static_assert(OCC * (SMEM + 2048) <= 228 * 1024, "over the shared memory of an SM");
};
constexpr int kMostCtas = 3, kMostRows = 2;              // of an SM, of a CTA, over all shapes

// Shuffled layout of a row's state: [FRAG][32 lanes] float4.  Fragment k NH + n
// holds channels of m tile k for heads 8n + 2t and 8n + 2t + 1 (the accumulator of
// an MMA), fragment KS NH + n the two maxima and this lane's two sums.
template <int D, bool E4M3, int NH>
struct State {
    static constexpr int KS = D / 16;
    float o[NH][KS][4], m[NH][2], l[NH][2];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][k][i] = 0.f;
        }
    }
    // fragment i of this lane
    __device__ __forceinline__ float4 frag(int i) const {
        const int n = i % NH, k = i / NH;
        return k < KS ? make_float4(o[n][k][0], o[n][k][1], o[n][k][2], o[n][k][3])
                      : make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
    }
    __device__ __forceinline__ void store(float4* to) const {   // to: this lane's
#pragma unroll
        for (int i = 0; i < (KS + 1) * NH; ++i) to[i * 32] = frag(i);
    }
    // Adds another state of the row; from(i): its fragment i of this lane.  (The
    // roundings are spelled out: all copies of this code give the same bits.)
    template <typename F>
    __device__ __forceinline__ void add(F from) {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const float4 z = from(KS * NH + n);
            const float zm[2] = {z.x, z.y}, zl[2] = {z.z, z.w};
            float mine[2], theirs[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float top = fmaxf(m[n][c], zm[c]);
                mine[c] = m[n][c] == top ? 1.f : ex2(m[n][c] - top);
                theirs[c] = zm[c] == -INFINITY ? 0.f : ex2(zm[c] - top);
                m[n][c] = top;
                l[n][c] = fmaf(theirs[c], zl[c], __fmul_rn(mine[c], l[n][c]));
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float4 y = from(k * NH + n);
                o[n][k][0] = fmaf(theirs[0], y.x, __fmul_rn(mine[0], o[n][k][0]));
                o[n][k][1] = fmaf(theirs[1], y.y, __fmul_rn(mine[1], o[n][k][1]));
                o[n][k][2] = fmaf(theirs[0], y.z, __fmul_rn(mine[0], o[n][k][2]));
                o[n][k][3] = fmaf(theirs[1], y.w, __fmul_rn(mine[1], o[n][k][3]));
            }
        }
    }
};

// Where a row's result goes, and the units of its O.
struct RowOut {
    long long at;      // row of q, o, lse: s HQ + first head
    int heads;         // of the block
    float unit;        // what a unit of V is worth (e4m3)
};

// Writes one fragment (m tile k, heads 8n + 2t + {0, 1}) of a finished row.
template <int D, bool E4M3>
__device__ __forceinline__ void write_frag(const PagedArgs& a, const RowOut& r, int n, int k,
                                           int g, int t, const float (&o)[4],
                                           const float (&by)[2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int head = 8 * n + 2 * t + c;
        if (head >= r.heads) continue;
        __nv_bfloat16* to = a.o + (r.at + head) * D + 16 * k;
        // rows g, g + 8 of the m tile are channels g, g + 8 (bf16) or 2g, 2g + 1
        if (E4M3) {
            *reinterpret_cast<uint32_t*>(to + 2 * g) =
                ptx::pack_bf16(o[c] * by[c], o[c + 2] * by[c]);
        } else {
            to[g] = __float2bfloat16_rn(o[c] * by[c]);
            to[g + 8] = __float2bfloat16_rn(o[c + 2] * by[c]);
        }
    }
}
// The factors of a finished row's O (heads 8n + 2t + c), and its lse.
template <bool E4M3>
__device__ __forceinline__ void finish_heads(const PagedArgs& a, const RowOut& r, int n, int g,
                                             int t, const float (&m)[2], float (&l)[2], bool lse,
                                             float (&by)[2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
        // (a sum of zero: nothing was seen.  The maximum would not tell it from NaN.)
        const bool any = l[c] != 0.f;
        const int head = 8 * n + 2 * t + c;
        by[c] = any ? r.unit / l[c] : 0.f;
        if (lse && a.lse && g == 0 && head < r.heads)
            a.lse[r.at + head] = any ? (m[c] + (lg2(l[c]) - kLow<E4M3>)) * kLn2 : -INFINITY;
    }
}

// Adds parts w, w + TW, ... of a row's `count` to st: part 0 lies at
// `first`, the others from `rest` on, `step` float4 apart.  B parts are on their
// way at once.
template <int B, int TW, int D, bool E4M3, int NH>
__device__ __forceinline__ void add_parts(State<D, E4M3, NH>& st, const float4* first,
                                          const float4* rest, int count, int step, int w,
                                          int lane) {
    constexpr int F = Shape<D, E4M3, NH>::FRAG;
#pragma unroll 1
    for (int i = w; i < count; i += B * TW) {
        float4 y[B][F];
#pragma unroll
        for (int e = 0; e < B; ++e) {
            const int j = i + e * TW;
            const float4* p = (j == 0 ? first : rest + (long long)(j - 1) * step) + lane;
#pragma unroll
            for (int k = 0; k < F; ++k)
                y[e][k] = j < count ? __ldcg(p + k * 32)
                                    : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        }
#pragma unroll
        for (int e = 0; e < B; ++e)
            if (i + e * TW < count) st.add([&](int k) { return y[e][k]; });
    }
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// WH rows (blocks of query heads) side by side, of TW warps each.
template <int D, bool E4M3, int NH, int WH>
__global__ void __launch_bounds__(kThreads, Shape<D, E4M3, NH>::OCC)
decode_kernel(const PagedArgs a, int HB, unsigned* __restrict__ tickets,
              float4* __restrict__ parts) {
    using Sh = Shape<D, E4M3, NH>;
    constexpr int KS = Sh::KS, TW = kWarps / WH;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ int s_seq;
    __shared__ long long s_at;
    __shared__ int s_last[WH];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int hs = warp / TW, tw = warp % TW;            // the warp's row, its place in it
    const int rows = a.HKV * HB / WH;                    // (groups of WH) rows of a sequence
    wait_for_previous();
    let_next_start();

    // ---- this CTA's stretch of the line of tiles ----
    const int per_thread = (a.S + kThreads - 1) / kThreads;
    const int s_lo = min(a.S, tid * per_thread), s_hi = min(a.S, s_lo + per_thread);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += make_span(a, seq_len(a, s)).slots<TW>();
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) s_scan[warp] = sum;
    if (tid < WH) s_last[tid] = 0;
    __syncthreads();
    long long before = sum - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    before *= rows;
    total *= rows;
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long begin = blockIdx.x * per, end = min(total, begin + per);
    if (begin >= end) return;
    if (mine > 0 && before <= begin && begin < before + mine * rows) {
        long long at = before;                           // the sequence that holds `begin`
        int s = s_lo;
        for (; s + 1 < s_hi; ++s) {
            const long long n = (long long)make_span(a, seq_len(a, s)).slots<TW>() * rows;
            if (begin < at + n) break;
            at += n;
        }
        s_seq = s;
        s_at = at;
    }
    __syncthreads();
    const uint32_t ring = ptx::smem_u32(smem) + warp * Sh::RING;
    // of the row's warps but the first
    float4* mail = reinterpret_cast<float4*>(smem + kWarps * Sh::RING) + lane +
                   hs * (TW - 1) * (Sh::FRAG * 32);
    const int gshift = a.page_shift - 4;                 // groups per page, log2

    // A stretch's piece of one row, as the warp sees it.
    struct Piece {
        int s, row, tile0, tile1, tiles;
        long long seq_at, at, next;                      // line index of its sequence, of itself,
                                                         // of what follows
        Span sp;
        int g0, steps;                                   // the warp's first group, groups
    };
    // p.s, p.seq_at, p.at are set; whether a piece begins there (or after the
    // end of a row that reaches into the stretch)
    auto enter = [&](Piece& p) {
        int len;
        for (;;) {
            if (p.at >= end) return false;
            p.sp = make_span(a, seq_len(a, p.s));
            len = p.sp.slots<TW>();
            while (p.at >= p.seq_at + (long long)len * rows && p.s + 1 < a.S) {
                p.seq_at += (long long)len * rows;
                p.sp = make_span(a, seq_len(a, ++p.s));
                len = p.sp.slots<TW>();
            }
            p.tiles = p.sp.tiles<TW>();
            p.row = (int)((p.at - p.seq_at) / len);
            p.tile0 = (int)((p.at - p.seq_at) % len);
            if (p.tile0 < p.tiles) break;
            p.at += len - p.tile0;                       // the row's last tiles were before
        }
        p.tile1 = (int)min((long long)p.tiles, p.tile0 + (end - p.at));
        p.next = p.at + (p.tile1 == p.tiles ? len - p.tile0 : p.tile1 - p.tile0);
        p.g0 = p.tile0 * TW + tw;
        const int g1 = min(p.sp.n, p.tile1 * TW);
        p.steps = p.g0 < g1 ? (g1 - p.g0 + TW - 1) / TW : 0;
        return true;
    };
    Piece in;                                            // being loaded
    in.s = s_seq;
    in.seq_at = s_at;
    in.at = begin;
    if (!enter(in)) return;
    Piece cur = in;                                      // being worked on

    // ---- loads: one step of the warp, or nothing, is one group of copies ----
    int in_step = 0, in_stage = 0;
    bool more = true;
    auto page_of = [&]() {
        return in_step < in.steps
                   ? __ldg(a.table + (size_t)in.s * a.max_pages +
                           (in.sp.group(in.g0 + in_step * TW) >> gshift))
                   : 0;
    };
    int page = page_of();
    auto issue = [&]() {
        while (in_step >= in.steps && more) {
            in.at = in.next;
            more = enter(in);
            if (!more) break;
            in_step = 0;
            page = page_of();
        }
        if (more && in_step < in.steps) {
            const int grp = in.sp.group(in.g0 + in_step * TW), j0 = grp * kGroup;
            const bool good = (unsigned)page < (unsigned)a.num_pages;
            if (!good) record();
            const long long off = (good ? page : 0) * a.page_stride +
                                  (grp & ((1 << gshift) - 1)) * kGroup * a.token_stride +
                                  ((in.row * WH + hs) / HB) * a.head_stride;
            const char* kp = static_cast<const char*>(a.kp) + off * (E4M3 ? 1 : 2);
            const char* vp = static_cast<const char*>(a.vp) + off * (E4M3 ? 1 : 2);
            const long long ts = a.token_stride * (E4M3 ? 1 : 2);
            const uint32_t st = ring + in_stage * (2 * Sh::TILE);
#pragma unroll
            for (int r = 0; r < Sh::TILE / 512; ++r) {
                const int x = r * 32 + lane, row_ = x / Sh::RC, c = x % Sh::RC;
                const int j = j0 + row_;
                const bool on = good && j < in.sp.len && (j >= in.sp.low || j < in.sp.sinks);
                // chunks are permuted within 128 bytes so that eight rows of
                // one chunk lie in different banks
                const int sw = Sh::RC >= 8 ? (row_ & 7) : ((row_ >> 1) & 3);
                const uint32_t d = st + row_ * Sh::RB + ((c ^ sw) << 4);
                const long long o = row_ * ts + c * 16;
                cp_async16_zfill(d, kp + o, on);
                cp_async16_zfill(d + Sh::TILE, vp + o, on);
            }
            ++in_step;
            in_stage = in_stage + 1 == Sh::STAGES ? 0 : in_stage + 1;
            page = page_of();
        }
        ptx::cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < Sh::STAGES - 1; ++i) issue();

    int stage = 0;
    for (bool first = true;; first = false) {
        const int u = cur.row * WH + hs, h = u / HB, hq0 = h * a.G + u % HB * (8 * NH);
        RowOut out;
        out.at = (long long)cur.s * a.HQ + hq0;
        out.heads = min(8 * NH, (h + 1) * a.G - hq0);
        out.unit = E4M3 && a.vs ? a.vs[h] : 1.f;

        // ---- Q as the B operand: head g (+ 8 n), channels of this lane ----
        // e4m3: q in fp16, the largest scaled by a power of two to [2^14, 2^15) (put
        // back into the logits' factor), so that channels down to 2^-31 of it are
        // exact; channel pairs in the order that a 32-bit piece of a K row gives
        // them.
        uint32_t qf[NH][KS][2];
        float f[NH][2];                                  // logit factors of heads 2t, 2t + 1
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const bool on = 8 * n + g < out.heads;
            const __nv_bfloat16* q = a.q + cur.s * a.q_stride + (long long)(hq0 + 8 * n + g) * D;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (E4M3) {
                    const uint2 x = on ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * t)
                                       : make_uint2(0, 0);
                    qf[n][k][0] = x.x;
                    qf[n][k][1] = x.y;
                } else {
                    qf[n][k][0] = on ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t) : 0;
                    qf[n][k][1] =
                        on ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t + 8) : 0;
                }
            }
            f[n][0] = f[n][1] = a.scale * kLog2e;
            if (E4M3) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = __bfloat1622float2(
                            *reinterpret_cast<const __nv_bfloat162*>(&qf[n][k][i]));
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // as far as 2^-e is a normal number
                const int e = max(-126, min(126, (int)(__float_as_uint(top) >> 23) - 127 - 14));
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = __bfloat1622float2(
                            *reinterpret_cast<const __nv_bfloat162*>(&qf[n][k][i]));
                        qf[n][k][i] = pack_f16(x.x * pow2i(-e), x.y * pow2i(-e));
                    }
                const float ks = a.ks ? a.ks[h] : 1.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    f[n][i] *= ks * pow2i(__shfl_sync(0xffffffffu, e, 4 * (2 * t + i)));
            }
        }

        State<D, E4M3, NH> st;
        st.clear();
        for (int i = 0; i < cur.steps; ++i) {
            cp_async_wait<Sh::STAGES - 2>();
            __syncwarp();                                // every lane's; the step before is read
            issue();
            const uint32_t kt = ring + stage * (2 * Sh::TILE), vt = kt + Sh::TILE;
            stage = stage + 1 == Sh::STAGES ? 0 : stage + 1;

            // ---- S^T = K Q^T, in two chains of sums ----
            float x[NH][4], y[NH][4];
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] = y[n][e] = 0.f;
            {
                const int r = lane & 15, up = lane >> 4;
                const int sw = Sh::RC >= 8 ? (r & 7) : ((r >> 1) & 3);
                if (!E4M3) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t af[4];
                        ldsm4(af, kt + r * Sh::RB + (((2 * k + up) ^ sw) << 4));
#pragma unroll
                        for (int n = 0; n < NH; ++n)
                            mma16816<false>(k & 1 ? y[n] : x[n], af, qf[n][k][0], qf[n][k][1]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        uint32_t c[4];
                        ldsm4(c, kt + r * Sh::RB + (((k + up) ^ sw) << 4));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t lo = c[2 * e], hi = c[2 * e + 1];
                            const uint32_t af[4] = {e4m3x2_f16x2((uint16_t)lo),
                                                    e4m3x2_f16x2((uint16_t)hi),
                                                    e4m3x2_f16x2((uint16_t)(lo >> 16)),
                                                    e4m3x2_f16x2((uint16_t)(hi >> 16))};
#pragma unroll
                            for (int n = 0; n < NH; ++n)
                                mma16816<true>(e ? y[n] : x[n], af, qf[n][k + e][0],
                                               qf[n][k + e][1]);
                        }
                    }
                }
            }

            // ---- weights ----
            const int j0 = cur.sp.group(cur.g0 + i * TW) * kGroup;
            const bool edge = j0 + kGroup > cur.sp.len || j0 < cur.sp.low;
            bool rise = false;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[n][e] = (x[n][e] + y[n][e]) * f[n][e & 1];
                    if (edge) {
                        const int j = j0 + g + 8 * (e >> 1);
                        if (!(j < cur.sp.len && (j >= cur.sp.low || j < cur.sp.sinks)))
                            x[n][e] = -INFINITY;
                    }
                    rise |= x[n][e] > st.m[n][e & 1] + 8.f;
                }
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(st.m[n][c], fmaxf(x[n][c], x[n][c + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float keep = st.m[n][c] == top ? 1.f : ex2(st.m[n][c] - top);
                        st.m[n][c] = top;
                        st.l[n][c] *= keep;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            st.o[n][k][c] *= keep;
                            st.o[n][k][c + 2] *= keep;
                        }
                    }
            }
            uint32_t pf[NH][2], pl[NH][2];               // weights (bf16: and what they lost)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float top = st.m[n][e & 1];
                    w[e] = ex2(x[n][e] - (top == -INFINITY ? 0.f : top) + kLow<E4M3>);
                }
                st.l[n][0] += w[0] + w[2];
                st.l[n][1] += w[1] + w[3];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float w0 = w[2 * e], w1 = w[2 * e + 1];
                    if (E4M3) {
                        pf[n][e] = movm_t(pack_f16(w0, w1));
                    } else {
                        const uint32_t p = ptx::pack_bf16(w0, w1);
                        pf[n][e] = movm_t(p);
                        pl[n][e] = movm_t(ptx::pack_bf16(w0 - __uint_as_float(p << 16),
                                                         w1 - __uint_as_float(p & 0xffff0000u)));
                    }
                }
            }

            // ---- O^T += V^T P ----
            if (!E4M3) {
                const int r = (lane & 7) + (lane >> 4) * 8, up = (lane >> 3) & 1;
                const int sw = r & 7;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t af[4];
                    ldsm4_t(af, vt + r * Sh::RB + (((2 * k + up) ^ sw) << 4));
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        mma16816<false>(st.o[n][k], af, pf[n][0], pf[n][1]);
                        mma16816<false>(st.o[n][k], af, pl[n][0], pl[n][1]);
                    }
                }
            } else {
                // a 16-bit unit is two channels of a token; lane g gets unit g of
                // two tokens, split here into the even and the odd channel
                const int r = lane & 15, up = lane >> 4;
                const int sw = Sh::RC >= 8 ? (r & 7) : ((r >> 1) & 3);
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t c[4];
                    ldsm4_t(c, vt + r * Sh::RB + (((k + up) ^ sw) << 4));
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t lo = __byte_perm(c[2 * e], 0, 0x3120);
                        const uint32_t hi = __byte_perm(c[2 * e + 1], 0, 0x3120);
                        const uint32_t af[4] = {e4m3x2_f16x2((uint16_t)lo),
                                                e4m3x2_f16x2((uint16_t)(lo >> 16)),
                                                e4m3x2_f16x2((uint16_t)hi),
                                                e4m3x2_f16x2((uint16_t)(hi >> 16))};
#pragma unroll
                        for (int n = 0; n < NH; ++n)
                            mma16816<true>(st.o[n][k + e], af, pf[n][0], pf[n][1]);
                    }
                }
            }
        }

        // ---- the end of the piece: the row's first warp collects ----
        const bool whole = cur.tile0 == 0 && cur.tile1 == cur.tiles;
        const long long row_at = cur.seq_at + (long long)cur.row * cur.sp.slots<TW>();
        const int c0 = (int)(row_at / per), c1 = (int)((row_at + cur.tiles - 1) / per);
        // the parts of the row: CTA c0 leaves its own in its second slot, the others in their
        // first
        Piece then = cur;
        then.at = cur.next;
        const bool last = !enter(then);
        constexpr int kPart = WH * Sh::FRAG * 32, kStep = 2 * kPart;   // float4 between slots, CTAs
        float4* slots = parts + (2LL * c0 + 1) * kPart + hs * (Sh::FRAG * 32);
        auto send = [&]() { st.store(mail + (tw - 1) * (Sh::FRAG * 32)); };
        auto collect = [&]() {
#pragma unroll 1
            for (int w = 0; w < TW - 1; ++w)
                st.add([&](int i) { return mail[(w * Sh::FRAG + i) * 32]; });
        };
        auto write = [&]() {
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                float by[2];
                finish_heads<E4M3>(a, out, n, g, t, st.m[n], st.l[n], true, by);
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    write_frag<D, E4M3>(a, out, n, k, g, t, st.o[n][k], by);
            }
        };
        if (tw > 0) {
            if (!first) bar_sync(2 + 2 * hs, 32 * TW);   // the first warp has read the last one
            send();
            bar_arrive(1 + 2 * hs, 32 * TW);
        } else {
            bar_sync(1 + 2 * hs, 32 * TW);
            collect();
            if (!last) bar_arrive(2 + 2 * hs, 32 * TW);
            if (whole) {
                write();
            } else {
                float4* slot = (int)blockIdx.x == c0
                                   ? slots
                                   : slots + kPart +
                                         (long long)((int)blockIdx.x - c0 - 1) * kStep;
                st.store(slot + lane);
                __threadfence();
                __syncwarp();
                unsigned ticket = 0;
                if (lane == 0) ticket = atomicAdd(tickets + c0 * WH + hs, 1u);
                ticket = __shfl_sync(0xffffffffu, ticket, 0);
                if (ticket == (unsigned)(c1 - c0)) {
                    __threadfence();
                    if (lane == 0) tickets[c0 * WH + hs] = 0;   // as the next call expects it
                    if (last) {
                        if (lane == 0) s_last[hs] = 1;   // the row's warps join it below
                    } else {
                        // alone, with the sums that the row's warps would take
                        st.clear();
                        add_parts<1, TW>(st, slots, slots + kPart, c1 - c0 + 1, kStep, 0, lane);
#pragma unroll 1
                        for (int w = 1; w < TW; ++w) {
                            State<D, E4M3, NH> more;
                            more.clear();
                            add_parts<1, TW>(more, slots, slots + kPart, c1 - c0 + 1, kStep, w,
                                             lane);
                            st.add([&](int i) { return more.frag(i); });
                        }
                        write();
                    }
                }
            }
        }
        if (last) {
            __syncthreads();
            bool any = false;
#pragma unroll
            for (int i = 0; i < WH; ++i) any |= s_last[i] != 0;
            if (any) {
                const bool mine_too = s_last[hs] != 0;
                if (mine_too) {
                    st.clear();
                    add_parts<NH == 1 ? 3 : 1, TW>(st, slots, slots + kPart, c1 - c0 + 1, kStep,
                                                   tw, lane);
                    if (tw > 0) send();
                }
                __syncthreads();
                if (mine_too && tw == 0) {
                    collect();
                    write();
                }
            }
            break;
        }
        cur = then;
    }
    cp_async_wait<0>();
}

// The workspace: a counter for each CTA and row, then two parts for each.
size_t tickets_bytes() {
    return align256((size_t)kMostRows * kMostCtas * sm_count() * sizeof(unsigned));
}

template <int D, bool E4M3, int NH, int WH>
kda_status launch_rows(const PagedArgs& a, void* ws, cudaStream_t s) {
    using Sh = Shape<D, E4M3, NH>;
    static bool set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
    auto* fn = decode_kernel<D, E4M3, NH, WH>;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Sh::SMEM) != cudaSuccess)
            return KDA_ERR_CUDA;
        set[dev] = true;
    }
    const int HB = (a.G + 8 * NH - 1) / (8 * NH), W = Sh::OCC * sm_count();
    const long long most = (long long)a.S * a.HKV * HB * ((a.cap + 63LL) / 64 + 1 + kRowEnd);
    TimedLaunch tl("paged_decode", s);
    return launch_overlapped(fn, (unsigned)(most < W ? most : W), kThreads, Sh::SMEM, s, a, HB,
                             static_cast<unsigned*>(ws),
                             reinterpret_cast<float4*>(static_cast<char*>(ws) + tickets_bytes()));
}

// One row per CTA, or two: K and V rows of 128 bytes or less come from HBM at
// 0.87 of the rate of longer pieces, so where the next head's rows lie beside
// them, both are taken at once.
template <int D, bool E4M3, int NH>
kda_status launch(const PagedArgs& a, void* ws, cudaStream_t s) {
    if constexpr (Shape<D, E4M3, NH>::RB <= 128) {
        const int HB = (a.G + 8 * NH - 1) / (8 * NH);
        if (a.head_stride == D && a.HKV * HB % 2 == 0) return launch_rows<D, E4M3, NH, 2>(a, ws, s);
    }
    return launch_rows<D, E4M3, NH, 1>(a, ws, s);
}

template <int D, bool E4M3, int NH>
size_t parts_bytes() {
    using Sh = Shape<D, E4M3, NH>;
    const size_t rows = Sh::RB <= 128 ? kMostRows : 1;
    return align256(rows * 2 * Sh::FRAG * 512 * Sh::OCC * sm_count());
}

}  // namespace

size_t paged_decode_ws_bytes(const PagedArgs& a, int D, bool e4m3) {
    size_t parts;
    if (D == 128 && a.G <= 8)
        parts = e4m3 ? parts_bytes<128, true, 1>() : parts_bytes<128, false, 1>();
    else if (D == 128)
        parts = e4m3 ? parts_bytes<128, true, 2>() : parts_bytes<128, false, 2>();
    else if (a.G <= 8)
        parts = e4m3 ? parts_bytes<64, true, 1>() : parts_bytes<64, false, 1>();
    else
        parts = e4m3 ? parts_bytes<64, true, 2>() : parts_bytes<64, false, 2>();
    return tickets_bytes() + parts;
}

kda_status paged_decode_launch(const PagedArgs& a, int D, bool e4m3, void* ws, cudaStream_t s) {
    // up to 8 query heads of a key head in one block of MMA columns, else 16
    if (D == 128) {
        if (a.G <= 8)
            return e4m3 ? launch<128, true, 1>(a, ws, s) : launch<128, false, 1>(a, ws, s);
        return e4m3 ? launch<128, true, 2>(a, ws, s) : launch<128, false, 2>(a, ws, s);
    }
    if (a.G <= 8) return e4m3 ? launch<64, true, 1>(a, ws, s) : launch<64, false, 1>(a, ws, s);
    return e4m3 ? launch<64, true, 2>(a, ws, s) : launch<64, false, 2>(a, ws, s);
}

int* paged_decode_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_decode_error) == cudaSuccess ? static_cast<int*>(p)
                                                                         : nullptr;
}

}  // namespace kda
