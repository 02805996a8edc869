// Attention of prompt tokens over a paged key-value cache: causal, with a
// sliding window and sinks, on the tensor cores (tcgen05 + TMEM + TMA).
//
// A CTA takes 256 query rows of one (sequence, key head) as two tiles A, B of
// 128.  A row is a (token, query head) pair, the G heads that share the key
// head side by side, so shared heads fill the MMA's M axis and every K and V
// tile is read once for all of them.  Per tile of 128 cached tokens:
//     S = Q K^T                  tcgen05, fp32 in TMEM, one thread per row reads it
//     P = exp2(f S - m + 7)      f = scale log2(e); back to TMEM over S, in halves
//     O += P V                   tcgen05, P from TMEM, V as it lies (MN-major)
// While the softmax of one tile runs, the tensor core works for the other.
//
// What bounds it: for every 128 x 256 block the four products take 2240 cycles
// of the tensor core as measured alone (70 for each 128 x 128 x 16), the 32768
// exponentials 1024 of the special function units.  A pair of tiles takes 2900
// cycles: a chain of S -> weights (1500) -> P V and the next S (1100) -> on to
// the softmax again (300) is longer than the tensor core's work.  A prompt of
// 8192 tokens, 16 heads over 4, D = 128: 206 us in a graph, 1335 TFLOP/s, 0.72 of the
// bf16 rate of cuBLAS; the first and the last tile of an item, which are
// slower, and the items' unequal lengths are the rest.
//
// Softmax.  The weights of a tile are taken against a reference m of the row,
// the largest logit of its first half tile; only when the weights of a half
// tile add up to more than 65000 is a larger logit looked for, m moved to it, O
// and the sum rescaled and the half weighed again.  (f S - m in one rounding: m is
// off by its own, which the weights of such tiles share.  Above 2^10 that would show
// beside those of other tiles; there the exponent is f (S - S of the reference), so
// equal keys weigh the same for logits of any size.)  So as a rule no maximum is
// taken at all, and weights stay inside the range of fp16.  Sums are fp32.  P enters
// the product with V in fp16, which rounds a weight by up to 2^-11, a small part of
// the output's own rounding (2^-8), at the rate of a bf16 one (which alone would
// round weights by as much as the output).  The reference weighs 2^7, so that only
// weights below 2^-21 of it leave fp16's normal range (and are rounded by up to 2^-32
// of it): a long tail behind one strong token would show it if the reference weighed
// 1.  That leaves 2^9 for larger logits: a prompt of 8192 tokens does not look
// more often (at 2^9 for the reference it does: 225 us against 209), a window's rows, which
// start from a few sinks, do (138 us against 132).
//
// K and V tiles arrive by TMA, one box per page, into rings of slots, and a
// warpgroup turns what is not ready for the products into it, in place:
// * V in bf16 to fp16, scaled by a power of two 2^-E: the first tile's largest
//   value then lies in [2^12, 2^13); a later tile with values of 2^16 or more
//   raises E in the same way, and the rows' O are rescaled as for a moved
//   reference.  So the largest value so far is 2^12 or more, and bf16 values,
//   exact in fp16 down to 2^-17, are exact down to 2^-29 of it (but for
//   magnitudes below 2^-117: E is -100 at least).
// * e4m3 codes of K and V to fp16, exactly.  Q then goes to fp16 too, every row
//   scaled by a power of two that its logits' factor gives back: its largest value lies in
//   [2^14, 2^15), and those down to 2^-31 of that are exact.
// * Infinities and NaN in V to zeros (e4m3: in tiles that not all rows see whole), since a
//   weight of 0 would not keep them from the rows that do not see their token; the rows
//   that do get them at the end.
// * V rows past the sequence's end (they may hold NaN) to zeros.  Pages that none
//   of the rows sees, and pages out of range, are asked for at a coordinate outside the
//   pool, which TMA fills with zeros.
//
// Roles: warps 0-3 softmax and output of tile A, 4-7 of B, warp 8 TMA, warp 9
// MMA, warps 12-15 the conversions.  Every wait is bounded; on expiry the error
// is recorded and the CTA unwinds.  With few query rows the cached tokens are
// split over several CTAs, whose parts a second kernel joins.
#include <algorithm>
#include <climits>
#include <mutex>

#include "kda_paged.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_paged_prefill_error = 0;   // a kda_status

namespace {

using namespace ptx;
using namespace paged;

constexpr int kTile = 128;                  // query rows and cached tokens of a tile
// four warpgroups of 128 registers a thread at launch, dealt out again by role
constexpr int kThreads = 512;
constexpr int kRegsSoftmax = 176, kRegsIssue = 80, kRegsConvert = 80;
static_assert(2 * kRegsSoftmax + kRegsIssue + kRegsConvert <= 4 * 128, "registers of the launch");
constexpr long long kTimeoutCycles = 4000000000LL;   // ~2 s
constexpr float kLow = 7.f;                 // log2 of the weight at the reference
constexpr float kMost = 65000.f;            // sum of half a tile's weights that calls for a look
constexpr float kFar = 1024.f;              // references up to here serve the usual path

__device__ __forceinline__ void record(kda_status code) {
    atomicCAS(&g_paged_prefill_error, 0, (int)code);
}

// Bounded mbarrier wait: gives up after the limit, or when another wait has.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    uint32_t it = 0;
    while (!mbar_try_wait(bar, parity)) {
        if ((++it & 255u) == 0) {
            if (*reinterpret_cast<volatile int*>(&g_paged_prefill_error) == KDA_ERR_TIMEOUT)
                return false;
            if (clock64() - t0 > kTimeoutCycles) {
                atomicExch(&g_paged_prefill_error, (int)KDA_ERR_TIMEOUT);
                return false;
            }
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity));
}
// Time-bounded only: for copies and MMAs that must end before the CTA does.
__device__ __forceinline__ void wait_bar_drain(uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kTimeoutCycles) return;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// One lane of the warp, the same every time.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
// MMAs and commits that only the elected lane issues.  The whole warp runs the
// code around them, so that descriptors are computed once per warp.
// Descriptors are given by their low words; the high one is the same for all.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// D (+)= A B^T, both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint32_t adesc,
                                       uint32_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(adesc), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader), "n"(kDescHigh)
        : "memory");
}
// The same with A in tensor memory (16-bit pairs, 8 columns per 16 of K).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                       uint32_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tmem_st16_nw(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}
// Whether `p` holds for any of the 128 converting threads (named barrier 1).
__device__ __forceinline__ bool any_convert(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)p)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// a, b <- f * a + c, f * b + c
__device__ __forceinline__ void fma2(float& a, float& b, float f, float c) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ void mul2(float& a, float& b, float f) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f));
}
// The n lowest bits.
__device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}
// 2^e for any e (0 or infinity out of range).
__device__ __forceinline__ float pow2any(int e) {
    const int h = max(-126, min(126, e / 2)), k = max(-126, min(126, e - e / 2));
    return pow2i(h) * pow2i(k);
}

template <int D>
struct Plan {
    static constexpr uint32_t SLOT = kTile * D * 2;           // a K or V tile
    static constexpr uint32_t HALF = kTile * 128;             // its 64-column half
    // V waits for its conversion, so its ring is the longer one
    static constexpr int KS = D == 128 ? 2 : 4, VS = D == 128 ? 3 : 4, SLOTS = KS + VS;
    static constexpr uint32_t OFF_Q = 0;                      // two tiles
    static constexpr uint32_t OFF_KV = 2 * SLOT;
    static constexpr uint32_t OFF_BAR = OFF_KV + SLOTS * SLOT;
    static constexpr uint32_t SMEM = OFF_BAR + 512 + 1024;    // + alignment slack
    static_assert(SMEM <= 232448, "over the shared memory of a CTA");
};
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;       // S_A, S_B, O_A, O_B: 128 each

struct Split {                 // parts of a row, one per CTA that works on it
    float* o;                  // [splits][T * HQ][D], unscaled sums
    float2* ml;                // [splits][T * HQ] maximum (log2), sum
    int* valid;                // whether cu_seqlens held, for the kernel that joins the parts
};

// The tiles of cached tokens that an item's rows see: those of the sinks, then
// those from the window's start to the last row's position.
struct Span {
    int nsink, first, n;
    __device__ __forceinline__ int tile(int i) const { return i < nsink ? i : i - nsink + first; }
};
__device__ __forceinline__ Span make_span(const PagedArgs& a, int p_min, int p_max) {
    Span s = {0, 0, 0};
    if (p_max < 0) return s;
    const int low = a.window ? max(0, p_min - a.window + 1) : 0;
    s.first = low / kTile;
    s.nsink = min((min(a.sinks, low) + kTile - 1) / kTile, s.first);
    s.n = s.nsink + p_max / kTile + 1 - s.first;
    return s;
}

// The infinities and NaN of V that a query at position p sees in tiles [t0, t1] of
// its span, in 32 channels: a bit per channel for +inf (x) and -inf (y), both for NaN.
// v: the head's row 0 of page 0, at the first of the channels.
template <bool E4M3>
__device__ __noinline__ uint2 not_finite(const char* v, const int* table, Span sp, int t0, int t1,
                                         int p, int window, int sinks, int page_shift,
                                         int num_pages, long long page_bytes,
                                         long long token_bytes) {
    uint2 r = make_uint2(0, 0);
    for (int t = t0; t <= t1; ++t) {
        const int j0 = sp.tile(t) * kTile;
        for (int j = j0; j < j0 + kTile && j <= p; ++j) {
            if (window && j <= p - window && j >= sinks) continue;
            const int page = table[j >> page_shift];
            if ((unsigned)page >= (unsigned)num_pages) continue;
            const uint4* row = reinterpret_cast<const uint4*>(
                v + page * page_bytes + (j & ((1 << page_shift) - 1)) * token_bytes);
#pragma unroll 1
            for (int c = 0; c < (E4M3 ? 2 : 4); ++c) {
                const uint4 y = row[c];
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < (E4M3 ? 16 : 8); ++e) {
                    if (E4M3) {
                        const bool nan = (w[e >> 2] >> 8 * (e & 3) & 0x7fu) == 0x7fu;
                        r.x |= (uint32_t)nan << (16 * c + e);
                        r.y |= (uint32_t)nan << (16 * c + e);
                    } else {
                        const uint32_t b = w[e >> 1] >> 16 * (e & 1) & 0xffffu;
                        const bool nan = (b & 0x7fffu) > 0x7f80u;
                        r.x |= (uint32_t)(nan || b == 0x7f80u) << (8 * c + e);
                        r.y |= (uint32_t)(nan || b == 0xff80u) << (8 * c + e);
                    }
                }
            }
        }
    }
    return r;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
               const PagedArgs a, int TB, int heads_first, Split part) {
    using P = Plan<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::OFF_BAR);
    // slots of K, then of V
    uint64_t* kv_full = bars;                     // [SLOTS] loaded
    uint64_t* kv_ready = kv_full + P::SLOTS;      // [SLOTS] converted
    uint64_t* kv_empty = kv_ready + P::SLOTS;     // [SLOTS]
    // slot of tile n, and the parity of its barriers
    auto k_slot = [](int n) { return n % P::KS; };
    auto v_slot = [](int n) { return P::KS + n % P::VS; };
    auto k_par = [](int n) { return (uint32_t)(n / P::KS) & 1; };
    auto v_par = [](int n) { return (uint32_t)(n / P::VS) & 1; };
    uint64_t* q_full = kv_empty + P::SLOTS;       // [2]
    uint64_t* q_ready = q_full + 2;               // [2] converted (e4m3)
    uint64_t* s_full = q_ready + 2;               // [2] S is in TMEM, and O up to the tile before
    uint64_t* p_full = s_full + 2;                // [2][2] half of P is in TMEM
    uint64_t* o_half = p_full + 4;                // [2] O holds the first half of the tile
    uint64_t* o_full = o_half + 2;                // [2] O is complete
    uint64_t* done = o_full + 2;                  // every MMA has ended (unwinding)
    int* v_exp = reinterpret_cast<int*>(done + 1);   // [SLOTS] E of the V tile in the slot
    int* v_top = v_exp + P::SLOTS;                // bits of a tile's largest |v|
    int* v_bad = v_top + 1;                       // [2] first, last tile with an infinity or NaN
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(v_bad + 2);
    __shared__ int s_scan[kThreads / 32], s_seq, s_block, s_cu[2], s_len;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- which item: sequence, block of 2 TB tokens (the last ones, with the
    // most to read, start first), key head ----
    const int h = blockIdx.x % a.HKV;
    if (tid == 8 * 32) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    {
        const int each = (a.S + kThreads - 1) / kThreads;
        const int lo = min(a.S, tid * each), hi = min(a.S, lo + each);
        bool bad = tid == 0 && (a.cu[0] != 0 || a.cu[a.S] != a.T);
        int mine = 0;
        const int len_lo = lo < hi ? a.lens[lo] : 0;         // on its way with the others
        for (int s = lo; s < hi; ++s) {
            const int n = a.cu[s + 1] - a.cu[s];
            bad |= n < 0 || a.cu[s] < 0 || a.cu[s + 1] > a.T;
            if (!bad) mine += (n + 2 * TB - 1) / (2 * TB);
        }
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_scan[warp] = sum;
        const bool refused = __syncthreads_or(bad);
        if (gridDim.y > 1 && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) *part.valid = !refused;
        if (refused) {
            if (tid == 0) record(KDA_ERR_SHAPE);
            return;
        }
        int before = sum - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        const int item = total - 1 - (int)(blockIdx.x / a.HKV);
        if (item < 0) return;
        if (item >= before && item < before + mine) {
            int s = lo, at = before;
            for (; s + 1 < hi; ++s) {
                const int n = (a.cu[s + 1] - a.cu[s] + 2 * TB - 1) / (2 * TB);
                if (item < at + n) break;
                at += n;
            }
            s_seq = s;
            s_block = item - at;
            s_cu[0] = a.cu[s];
            s_cu[1] = a.cu[s + 1];
            s_len = s == lo ? len_lo : a.lens[s];
        }
    }
    if (tid == 10 * 32) {
        for (int i = 0; i < P::SLOTS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_ready[i], kTile);
            mbar_init(&kv_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&q_ready[x], kTile);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[2 * x], kTile);
            mbar_init(&p_full[2 * x + 1], kTile);
            mbar_init(&o_half[x], 1);
            mbar_init(&o_full[x], 1);
        }
        mbar_init(done, 1);
        *v_top = 0;
        v_bad[0] = INT_MAX;
        v_bad[1] = -1;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_holder, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int s = s_seq, cu0 = s_cu[0], nq = s_cu[1] - cu0;
    int len = s_len;
    if (len < 0 || len > a.cap) {
        if (tid == 0) record(KDA_ERR_SHAPE);
        len = 0;
    }
    const int i0 = s_block * 2 * TB;                         // first token of tile A in the prompt
    const int p0 = len - nq + i0;                            // its position
    const int p_last = min(p0 + 2 * TB, len) - 1;
    const Span sp = make_span(a, p0, p_last);
    const int n_lo = (int)((long long)sp.n * blockIdx.y / gridDim.y);
    const int n_hi = (int)((long long)sp.n * (blockIdx.y + 1) / gridDim.y);
    const int N = n_hi - n_lo;                               // tiles of this CTA

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == 8 && N > 0) {
            // ---------------- TMA ----------------
            if (lane == 0) {
                for (int x = 0; x < 2; ++x) {
                    mbar_arrive_expect_tx(&q_full[x], (uint32_t)(TB * a.G * D * 2));
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(smem + P::OFF_Q + x * P::SLOT + c * P::HALF, &tm_q, &q_full[x],
                                    64 * c, h * a.G, cu0 + i0 + x * TB);
                }
            }
            const int rows = min(1 << a.page_shift, kTile);  // rows of a box
            const int boxes = kTile / rows;
            const int* table = a.table + (size_t)s * a.max_pages;
            const int low = a.window ? p0 - a.window + 1 : 0;    // first token of the window
            int issued = 0;
            for (int n = 0; n < N; ++n) {
                const int j0 = sp.tile(n_lo + n) * kTile;
                int page = a.num_pages;                      // outside the pool: zeros
                const int j = j0 + lane * rows;
                // (pages that none of the rows sees may have been given back)
                if (lane < boxes && j <= p_last && (j + rows > low || j < a.sinks)) {
                    page = __ldg(table + (j >> a.page_shift));
                    if ((unsigned)page >= (unsigned)a.num_pages) {
                        record(KDA_ERR_SHAPE);
                        page = a.num_pages;
                    }
                }
                const int r0 = j & ((1 << a.page_shift) - 1);
                const int y = heads_first ? r0 : h, z = heads_first ? h : r0;
                bool ok = true;
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = kv ? v_slot(n) : k_slot(n);
                    ok = wait_bar_warp(&kv_empty[slot], (kv ? v_par(n) : k_par(n)) ^ 1);
                    if (!ok) break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&kv_full[slot], E4M3 ? P::SLOT / 2 : P::SLOT);
                    __syncwarp();
                    if (lane < boxes) {
                        const CUtensorMap* map = kv ? &tm_v : &tm_k;
                        uint8_t* dst = smem + P::OFF_KV + slot * P::SLOT;
                        if (E4M3) {
                            tma_load_4d(dst + lane * rows * D, map, &kv_full[slot], 0, y, z, page);
                        } else {
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_4d(dst + lane * rows * 128 + c * P::HALF, map,
                                            &kv_full[slot], 64 * c, y, z, page);
                        }
                    }
                    issued = 2 * n + kv + 1;
                }
                if (!ok) break;
            }
            if (issued < 2 * N) {                            // unwinding: let the copies land
                for (int q = max(0, issued - 2 * P::SLOTS); q < issued; ++q) {
                    const int n = q >> 1, kv = q & 1;
                    // (of a slot's copies the last one)
                    if (2 * (n + (kv ? P::VS : P::KS)) + kv < issued) continue;
                    wait_bar_drain(&kv_full[kv ? v_slot(n) : k_slot(n)], kv ? v_par(n) : k_par(n));
                }
                for (int x = 0; x < 2; ++x) wait_bar_drain(&q_full[x], 0);
            }
            __syncwarp();
        } else if (warp == 9 && N > 0) {
            // ---------------- MMA ----------------
            const uint32_t leader = elect_one();
            constexpr uint32_t kF16 = ~((1u << 7) | (1u << 10));   // both operands fp16
            constexpr uint32_t ID_S = idesc_bf16_f32(kTile, kTile) & (E4M3 ? kF16 : ~0u);
            constexpr uint32_t ID_O = (idesc_bf16_f32(kTile, D) & kF16) | kBMajorMN;
            uint64_t* k_bar = E4M3 ? kv_ready : kv_full;
            uint64_t* q_bar = E4M3 ? q_ready : q_full;
            // descriptors: the address field counts 16 bytes
            const uint32_t qd = (uint32_t)sdesc_sw128(smem_u32(smem + P::OFF_Q));
            const uint32_t kd = (uint32_t)sdesc_sw128(smem_u32(smem + P::OFF_KV));
            const uint32_t vd = (uint32_t)sdesc_mn_sw128(smem_u32(smem + P::OFF_KV), P::HALF);
            auto s_mma = [&](int x, int slot) {
                const uint32_t qx = qd + x * (P::SLOT / 16), kx = kd + slot * (P::SLOT / 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = ((k >> 2) * P::HALF + (k & 3) * 32) / 16;
                    mma_ss(leader, tmem + TM_S + x * kTile, qx + o, kx + o, ID_S, k > 0);
                }
                commit(leader, &s_full[x]);
            };
            bool ok = wait_bar_warp(&q_bar[0], 0) && wait_bar_warp(&k_bar[0], 0);
            if (ok) {
                tc_fence_after();
                s_mma(0, 0);
                ok = wait_bar_warp(&q_bar[1], 0);
            }
            if (ok) {
                tc_fence_after();
                s_mma(1, 0);
                commit(leader, &kv_empty[0]);
            }
            for (int n = 0; n < N && ok; ++n) {
                const int vslot = v_slot(n), kslot = k_slot(n + 1);
                const uint32_t vx = vd + vslot * (P::SLOT / 16);
                ok = wait_bar_warp(&kv_ready[vslot], v_par(n));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    for (int e = 0; e < 2; ++e) {
                        ok = ok && wait_bar_warp(&p_full[2 * x + e], n & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k)
                            mma_ts(leader, tmem + TM_O + x * kTile,
                                   tmem + TM_S + x * kTile + 32 * e + 8 * k,
                                   vx + (4 * e + k) * (2048 / 16), ID_O, n > 0 || e > 0 || k > 0);
                        if (e == 0) commit(leader, &o_half[x]);
                    }
                    if (!ok) break;
                    if (x == 1) commit(leader, &kv_empty[vslot]);
                    if (n + 1 == N) {
                        commit(leader, &o_full[x]);
                    } else {
                        if (x == 0) ok = wait_bar_warp(&k_bar[kslot], k_par(n + 1));
                        if (!ok) break;
                        s_mma(x, kslot);
                        if (x == 1) commit(leader, &kv_empty[kslot]);
                    }
                }
            }
            if (!ok) {                                       // unwinding: let the MMAs end
                commit(leader, done);
                wait_bar_drain(done, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
        // ---------------- conversions ----------------
        const int t = tid & 127;
        bool ok = true;
        int E = 0;
        auto note_bad = [&](int n) {
            atomicMin(v_bad, n);
            atomicMax(v_bad + 1, n);
        };
        for (int n = 0; n < N; ++n) {
            const int j0 = sp.tile(n_lo + n) * kTile, valid = len - j0;   // rows of the sequence
            if (E4M3) {
                // A tile's codes fill the first half of its slot.  Lane groups of
                // D / 16 read a row; every 16 codes become two 16-byte chunks.
                constexpr int C = D / 16, R = 128 / C, L = kTile / R;
                const int c = t % C, r0 = t / C;
                // Do all rows see all of it?  Then they all get its NaN codes; else
                // these are looked for (in every tile: 148 us for 141 of the window case).
                const bool mixed = !(j0 + kTile - 1 <= p0 &&
                                     (a.window == 0 || j0 > p0 + 2 * TB - 1 - a.window));
                for (int kv = 0; kv < 2; ++kv) {
                    const int slot = kv ? v_slot(n) : k_slot(n);
                    uint8_t* tile = smem + P::OFF_KV + slot * P::SLOT;
                    ok = ok && wait_bar_warp(&kv_full[slot], kv ? v_par(n) : k_par(n));
                    if (kv && mixed) {
#pragma unroll 1
                        for (int r = r0; r < min(kTile, valid); r += R) {
                            uint32_t* w = reinterpret_cast<uint32_t*>(tile + r * D + c * 16);
                            // the low bits of a NaN code are all ones
                            auto ones = [](uint32_t y) { return (y & 0x7f7f7f7fu) + 0x01010101u; };
                            const uint4 y = *reinterpret_cast<const uint4*>(w);
                            const uint32_t any = ones(y.x) | ones(y.y) | ones(y.z) | ones(y.w);
                            if ((any & 0x80808080u) == 0) continue;
#pragma unroll 1
                            for (int e = 0; e < 4; ++e)
                                w[e] &= ~((ones(w[e]) >> 7 & 0x01010101u) * 0xffu);
                            note_bad(n);
                        }
                    }
                    uint4 x[L];
#pragma unroll
                    for (int i = 0; i < L; ++i) {
                        const int r = r0 + i * R;
                        x[i] = *reinterpret_cast<const uint4*>(tile + r * D + c * 16);
                        if (r >= valid) x[i] = make_uint4(0, 0, 0, 0);
                    }
                    any_convert(false);                      // all codes are read
                    if (!ok) continue;
#pragma unroll
                    for (int i = 0; i < L; ++i) {
                        const int r = r0 + i * R;
                        uint8_t* half = tile + (c >> 2) * P::HALF + r * 128;
                        const uint4 lo = make_uint4(e4m3x2_f16x2((uint16_t)x[i].x),
                                                    e4m3x2_f16x2((uint16_t)(x[i].x >> 16)),
                                                    e4m3x2_f16x2((uint16_t)x[i].y),
                                                    e4m3x2_f16x2((uint16_t)(x[i].y >> 16)));
                        const uint4 hi = make_uint4(e4m3x2_f16x2((uint16_t)x[i].z),
                                                    e4m3x2_f16x2((uint16_t)(x[i].z >> 16)),
                                                    e4m3x2_f16x2((uint16_t)x[i].w),
                                                    e4m3x2_f16x2((uint16_t)(x[i].w >> 16)));
                        // the upper lanes store their second chunk first: eight
                        // lanes then write eight different banks
                        const int k = 2 * (c & 3), first = c >> 2;
                        *reinterpret_cast<uint4*>(half + (((k + first) ^ (r & 7)) << 4)) =
                            first ? hi : lo;
                        *reinterpret_cast<uint4*>(half + (((k + 1 - first) ^ (r & 7)) << 4)) =
                            first ? lo : hi;
                    }
                    fence_async_smem();
                    mbar_arrive(&kv_ready[slot]);
                }
            } else {
                constexpr int L = D / 8;                     // 16-byte chunks of a thread
                const int slot = v_slot(n);
                uint8_t* tile = smem + P::OFF_KV + slot * P::SLOT;
                ok = ok && wait_bar_warp(&kv_full[slot], v_par(n));
                uint8_t* mine = tile + t * 16;               // chunk i lies 2048 i further
                const int rows = valid - t / 8;              // 16 (i mod 8) < rows: in the sequence
                // the tile's largest |v|, by the bits of pairs
                uint32_t top = 0;
                auto larger = [&](uint32_t w) {
                    const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&w);
                    const __nv_bfloat162 z =
                        __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top), __habs2(y));
                    top = *reinterpret_cast<const uint32_t*>(&z);
                };
#pragma unroll 8
                for (int i = 0; i < L; ++i) {
                    const uint4 y = *reinterpret_cast<const uint4*>(mine + i * 2048);
                    if (16 * (i & 7) < rows) {
                        larger(y.x);
                        larger(y.y);
                        larger(y.z);
                        larger(y.w);
                    }
                }
                top = max(top & 0xffffu, top >> 16);         // a bf16 without its sign
                // Does it fit at the scale as it stands?  The first tile sets the scale.
                const uint32_t most = (uint32_t)max(0, min(0xff, 127 + 16 + E)) << 7;
                if (n == 0 || any_convert(top >= most)) {
                    // the largest of the finite ones; the others become zeros
                    uint32_t big = top;
                    if (__builtin_expect(top >= 0x7f80u, 0)) {
                        big = 0;
#pragma unroll 1
                        for (int i = 0; i < 4 * L; ++i) {
                            if (16 * ((i >> 2) & 7) >= rows) continue;
                            uint32_t* at =
                                reinterpret_cast<uint32_t*>(mine + (i >> 2) * 2048 + (i & 3) * 4);
                            uint32_t w = *at;
                            if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                            if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
                            *at = w;
                            big = max(big, max(w & 0x7fffu, w >> 16 & 0x7fffu));
                        }
                    }
                    big = __reduce_max_sync(0xffffffffu, big);
                    if (lane == 0) atomicMax(v_top, (int)big);
                    if (top >= 0x7f80u) note_bad(n);
                    any_convert(false);
                    const int bits = *reinterpret_cast<volatile int*>(v_top);
                    const int want = max(-100, (bits >> 7) - 127 - 12);
                    any_convert(false);                      // all have read it
                    if (t == 0) *v_top = 0;                  // seen by the next tile's any_convert
                    E = n == 0 ? want : max(E, want);
                }
                const float down = pow2any(-E);
                if (!ok) continue;
#pragma unroll 8
                for (int i = 0; i < L; ++i) {
                    uint4 y = *reinterpret_cast<const uint4*>(mine + i * 2048);
                    uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v0 = __uint_as_float(w[e] << 16);
                        float v1 = __uint_as_float(w[e] & 0xffff0000u);
                        mul2(v0, v1, down);
                        w[e] = 16 * (i & 7) < rows ? pack_f16(v0, v1) : 0;
                    }
                    *reinterpret_cast<uint4*>(mine + i * 2048) = y;
                }
                if (t == 0) v_exp[slot] = E;
                fence_async_smem();
                mbar_arrive(&kv_ready[slot]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------- softmax and output: one thread per query row ----------------
        const int x = warp >> 2, r = tid & 127;
        const int i = i0 + x * TB + r / a.G;
        const bool live = r < TB * a.G && i < nq;
        const int p = min(len - nq + i, len - 1);            // (a dead row goes along)
        float f = a.scale * kLog2e;
        const int px = p0 + x * TB;                          // positions of the tile's rows
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + TM_S + x * kTile + lanes, to = tmem + TM_O + x * kTile + lanes;
        // the reference as a logit and as it stands in S (a dead row asks for nothing)
        float m = live ? -INFINITY : 0.f, s_ref = 0.f, l = 0.f;
        bool ok = true;
        int E = 0;
        if (E4M3 && N > 0) {
            ok = wait_bar_warp(&q_full[x], 0);
            uint8_t* q = smem + P::OFF_Q + x * P::SLOT + r * 128;
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 y = *reinterpret_cast<const uint4*>(q + (c >> 3) * P::HALF +
                                                                ((c & 7) ^ (r & 7)) * 16);
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    big = max3(big, fabsf(__uint_as_float(w[e] << 16)),
                               fabsf(__uint_as_float(w[e] & 0xffff0000u)));
            }
            // the largest to [2^14, 2^15), as far as 2^-e is a normal number
            const int e2 = max(-126, min(126, (__float_as_int(big) >> 23) - 127 - 14));
            const float down = pow2i(-e2);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                uint4* y = reinterpret_cast<uint4*>(q + (c >> 3) * P::HALF +
                                                    ((c & 7) ^ (r & 7)) * 16);
                uint4 z = *y;
                uint32_t* w = reinterpret_cast<uint32_t*>(&z);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = pack_f16(__uint_as_float(w[e] << 16) * down,
                                    __uint_as_float(w[e] & 0xffff0000u) * down);
                *y = z;
            }
            f *= pow2i(e2) * (a.ks ? a.ks[h] : 1.f);
            fence_async_smem();
            mbar_arrive(&q_ready[x]);
        }
        // every visible token weighs the same: 2^0 for any logit, and -infinity stays
        if (f == 0.f) f = 1e-37f;
        if (!live) f = 0.f;                                  // whatever its row of Q holds
        for (int n = 0; n < N && ok; ++n) {
            const int j0 = sp.tile(n_lo + n) * kTile;
            int Ev = E;
            if (!E4M3 && n > 0) {                            // the scale of this tile's V
                ok = wait_bar_warp(&kv_ready[v_slot(n)], v_par(n));
                Ev = v_exp[v_slot(n)];
            }
            ok = ok && wait_bar_warp(&s_full[x], n & 1);
            if (!ok) break;
            tc_fence_after();
            // every row of the tile sees all of it?
            const bool edge = !(j0 + kTile - 1 <= px &&
                                (a.window == 0 || j0 > px + TB - 1 - a.window));
            // Half a tile at a time: weights exp2(f S - m) against the reference m
            // as it stands, if that is all there is to do.
            auto weigh = [&](float (&v)[2][32], uint32_t (&w)[2][16], float add) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        fma2(v[c][2 * e], v[c][2 * e + 1], f, add);
                        const float w0 = ex2(v[c][2 * e]), w1 = ex2(v[c][2 * e + 1]);
                        add2(part[2 * (e & 1)], part[2 * (e & 1) + 1], w0, w1);
                        w[c][e] = pack_f16(w0, w1);
                    }
                return (part[0] + part[1]) + (part[2] + part[3]);
            };
            auto hand_over = [&](int e2, const uint32_t (&w)[2][16]) {
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_st16_nw(ts + 32 * e2 + 16 * c, w[c]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[2 * x + e2]);
            };
            int e2 = 0;
            bool look = false;
            if (!edge && Ev == E && !__any_sync(0xffffffffu, !(fabsf(m) < kFar))) {
                float v[2][2][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32_nw(ts + 32 * c, v[c >> 1][c & 1]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait_ld_dep(v[c >> 1][c & 1]);
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    uint32_t w[2][16];
                    const float sum = weigh(v[i2], w, kLow - m);
                    look = __any_sync(0xffffffffu, sum > kMost);
                    if (look) break;
                    l += sum;
                    hand_over(i2, w);
                    ++e2;
                }
            }
            // Else, at the second round at the latest, every row looks at its
            // largest logit, and takes it for reference if it is larger than the one it
            // has; S stays in TMEM until then.  The exponents are differences of logits,
            // so that the largest weight is 2^7 for logits of any size.
#pragma unroll 1
            for (; e2 < 2; ++e2) {
                float sum, keep = 1.f;
                uint32_t w[2][16];
                look = look || __any_sync(0xffffffffu, m == -INFINITY);
                for (;;) {
                    float v[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld32_nw(ts + 64 * e2 + 32 * c, v[c]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_wait_ld_dep(v[c]);
                    if (edge) {
                        const int hi = p + 1 - j0 - 64 * e2;
                        const int lo = a.window ? p - a.window + 1 - j0 - 64 * e2 : 0;
                        const int sk = a.sinks - j0 - 64 * e2;
                        const float none = f < 0.f ? INFINITY : -INFINITY;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t seen = below(hi - 32 * c) &
                                                  (~below(lo - 32 * c) | below(sk - 32 * c));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) v[c][e] = none;
                        }
                    }
                    if (look) {
                        float hi = v[0][0], lo = v[0][0];
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                hi = max3(hi, v[c][e], v[c][e + 1]);
                                lo = min3(lo, v[c][e], v[c][e + 1]);
                            }
                        // (larger in S: the products may round to the same number)
                        const float s_top = f < 0.f ? lo : hi, top = s_top * f;
                        const float rise = (s_top - s_ref) * f;
                        if (m == -INFINITY ? top > -INFINITY : rise > 0.f) {
                            keep = m == -INFINITY ? 0.f : ex2(-rise);
                            m = top;
                            s_ref = s_top;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            add2(v[c][e], v[c][e + 1], -s_ref, -s_ref);
                    sum = weigh(v, w, kLow);
                    if (look) break;
                    look = __any_sync(0xffffffffu, sum > kMost);
                    if (!look) break;
                }
                look = false;
                l = l * keep + sum;
                if (__builtin_expect(Ev != E, 0)) {
                    keep *= pow2any(E - Ev);
                    E = Ev;
                }
                const bool change = __any_sync(0xffffffffu, keep != 1.f);
                if (change && (n > 0 || e2 > 0)) {
                    // O must hold the half before
                    if (e2 > 0) {
                        ok = wait_bar_warp(&o_half[x], n & 1);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(to + 32 * c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= keep;
                        tmem_st32_nw(to + 32 * c, o);
                    }
                }
                // the first tile's scale, before its slot can be filled again (a warp
                // that does not come here has no row to write)
                if (!E4M3 && n == 0 && e2 == 1) {
                    ok = wait_bar_warp(&kv_ready[v_slot(0)], v_par(0));
                    E = v_exp[v_slot(0)];
                }
                hand_over(e2, w);
            }
        }
        // ---- output ----
        if (N > 0) {
            // (the last V tile's conversion: v_bad is as it stays)
            ok = ok && wait_bar_warp(&kv_ready[v_slot(N - 1)], v_par(N - 1)) &&
                 wait_bar_warp(&o_full[x], 0);
            tc_fence_after();
        }
        const int last_bad = N > 0 && ok && live ? v_bad[1] : -1;
        const long long row = ((long long)cu0 + i) * a.HQ + h * a.G + r % a.G;
        const bool any = l != 0.f;                           // 0: nothing was seen (NaN is not 0)
        const float back = pow2i(-(int)kLow);                // to weights of 1 at the reference
        l *= back;
        const bool split = gridDim.y > 1;
        const long long at = (long long)blockIdx.y * a.T * a.HQ + row;
        // O is in units of 2^E and of the head's scale
        const float unit = (E4M3 ? (a.vs ? a.vs[h] : 1.f) : pow2any(E)) * back;
        const float by = any ? (split ? unit : unit / l) : 0.f;
        // A whole tile leaves through shared memory (Q's, which is read) by one TMA
        // store: rows of 256 bytes, where a thread alone would write 16 at a time.
        const bool whole = !split && i0 + (x + 1) * TB <= nq;
        uint8_t* stage = smem + P::OFF_Q + x * P::SLOT + r * 128;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float o[32];
            if (N > 0 && ok) {
                tmem_ld32(to + 32 * c, o);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
            if (live && split) {
                if (any)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(part.o + at * D + 32 * c + 4 * e) = make_float4(
                            by * o[4 * e], by * o[4 * e + 1], by * o[4 * e + 2], by * o[4 * e + 3]);
            } else if (live) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (any)
                        w = make_uint4(pack_bf16(o[8 * e] * by, o[8 * e + 1] * by),
                                       pack_bf16(o[8 * e + 2] * by, o[8 * e + 3] * by),
                                       pack_bf16(o[8 * e + 4] * by, o[8 * e + 5] * by),
                                       pack_bf16(o[8 * e + 6] * by, o[8 * e + 7] * by));
                    const int k = 4 * c + e;                 // 16-byte chunk of the row
                    if (whole)
                        *reinterpret_cast<uint4*>(stage + (k >> 3) * P::HALF +
                                                  (((k & 7) ^ (r & 7)) << 4)) = w;
                    else
                        *reinterpret_cast<uint4*>(a.o + row * D + 8 * k) = w;
                }
            }
            __syncwarp();                                    // together into the next load
        }
        // the infinities and NaN that the row sees, in place of what was summed
        if (__builtin_expect(last_bad >= 0, 0)) {
            constexpr int B = E4M3 ? 1 : 2;                  // bytes of an element
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                const uint2 y = not_finite<E4M3>(
                    static_cast<const char*>(a.vp) + (h * a.head_stride + 32 * c) * B,
                    a.table + (size_t)s * a.max_pages, sp, n_lo + v_bad[0], n_lo + last_bad, p,
                    a.window, a.sinks, a.page_shift, a.num_pages, a.page_stride * B,
                    a.token_stride * B);
                for (uint32_t left = y.x | y.y; left != 0; left &= left - 1) {
                    const int e = __ffs(left) - 1, d = 32 * c + e;
                    // (a NaN that the sum has by itself, of a NaN weight, stays)
                    const float v = !(l == l) || (y.x & y.y) >> e & 1 ? NAN
                                    : y.x >> e & 1                    ? INFINITY
                                                                      : -INFINITY;
                    if (split)
                        part.o[at * D + d] = v;
                    else if (whole)
                        *reinterpret_cast<__nv_bfloat16*>(
                            stage + (d >> 6) * P::HALF + (((d >> 3 & 7) ^ (r & 7)) << 4) +
                            (d & 7) * 2) = __float2bfloat16_rn(v);
                    else
                        a.o[row * D + d] = __float2bfloat16_rn(v);
                }
            }
        }
        __syncwarp();                                        // (not every lane was there)
        if (whole) {
            fence_async_smem();
            asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + x) : "memory");
            if (r == 0) {
                for (int c = 0; c < D / 64; ++c)
                    tma_store_3d(&tm_o, stage + c * P::HALF, 64 * c, h * a.G, cu0 + i0 + x * TB);
                bulk_commit_group();
                bulk_wait_read_all();
            }
        }
        if (live && split) part.ml[at] = make_float2(m, l);
        if (live && !split && a.lse) a.lse[row] = any ? (m + lg2(l)) * kLn2 : -INFINITY;
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, TM_COLS);
}

// Joins the parts of a row: one warp per row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const PagedArgs a, Split part, int splits) {
    constexpr int E = D / 32;
    const long long rows = (long long)a.T * a.HQ;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows || *part.valid == 0) return;
    float top = -INFINITY;
    for (int k = 0; k < splits; ++k) top = fmaxf(top, part.ml[k * rows + row].x);
    float l = 0.f, o[E] = {};
    for (int k = 0; k < splits; ++k) {
        const float2 ml = part.ml[k * rows + row];
        if (ml.y == 0.f) continue;                           // nothing seen (but NaN is not 0)
        const float w = ex2(ml.x - top);
        l += w * ml.y;
        const float* src = part.o + (k * rows + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += w * src[e];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(a.o + row * D + lane * E + e) =
            pack_bf16(o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (top + lg2(l)) * kLn2;
}

// ---- host ----
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn get_encoder() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}
// bf16 tiles in the 128-byte swizzle, or codes as they lie.
bool encode(CUtensorMap* m, bool codes, const void* ptr, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return get_encoder()(m,
                         codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         rank, const_cast<void*>(ptr), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query tokens of a 128-row tile, and upper bounds of the items of a call.
int tile_tokens(const PagedArgs& a) { return kTile / a.G; }
long long most_items(const PagedArgs& a) {
    return ((long long)a.T / (2 * tile_tokens(a)) + std::min(a.S, a.T)) * a.HKV;
}
// CTAs per item: enough for the SMs when the items are few.
int most_splits(const PagedArgs& a) {
    return (int)std::max(1LL, std::min(32LL, sm_count() / most_items(a)));
}
size_t part_bytes(const PagedArgs& a, int D, int splits) {
    return align256((size_t)splits * a.T * a.HQ * D * sizeof(float));
}
size_t ml_bytes(const PagedArgs& a, int splits) {
    return align256((size_t)splits * a.T * a.HQ * sizeof(float2));
}

template <int D, bool E4M3>
kda_status launch(const PagedArgs& a, void* ws, cudaStream_t s) {
    static bool set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
    if (!get_encoder()) return KDA_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(prefill_kernel<D, E4M3>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Plan<D>::SMEM) != cudaSuccess)
            return KDA_ERR_CUDA;
        set[dev] = true;
    }
    const int TB = tile_tokens(a), page = 1 << a.page_shift;
    CUtensorMap mq, mk, mv, mo;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.HQ, (cuuint64_t)a.T};
        const cuuint64_t strides[2] = {
            (cuuint64_t)D * 2, (cuuint64_t)(a.T > 1 ? a.q_stride : (long long)a.HQ * D) * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)TB};
        const cuuint64_t dense[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.HQ * D * 2};
        if (!encode(&mq, false, a.q, 3, dims, strides, box) ||
            !encode(&mo, false, a.o, 3, dims, dense, box))
            return KDA_ERR_CUDA;
    }
    // heads and rows of a page in the order of their strides
    const bool hf = a.HKV > 1 && a.head_stride > a.token_stride;
    {
        const cuuint64_t size = E4M3 ? 1 : 2, row = (cuuint64_t)a.token_stride * size;
        const cuuint64_t head = (cuuint64_t)(a.HKV > 1 ? a.head_stride : D) * size;
        const cuuint64_t pg = a.num_pages > 1 ? (cuuint64_t)a.page_stride * size : row * page;
        const cuuint32_t rows = (cuuint32_t)std::min(page, kTile);
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(hf ? page : a.HKV),
                                    (cuuint64_t)(hf ? a.HKV : page), (cuuint64_t)a.num_pages};
        const cuuint64_t strides[3] = {hf ? row : head, hf ? head : row, pg};
        const cuuint32_t box[4] = {E4M3 ? (cuuint32_t)D : 64, hf ? rows : 1, hf ? 1 : rows, 1};
        if (!encode(&mk, E4M3, a.kp, 4, dims, strides, box) ||
            !encode(&mv, E4M3, a.vp, 4, dims, strides, box))
            return KDA_ERR_CUDA;
    }
    // a split takes four tiles or more of the longest row
    const int splits = (int)std::max<long long>(
        1, std::min<long long>(most_splits(a), a.cap / (4 * kTile)));
    char* w = static_cast<char*>(ws);
    const Split part = {static_cast<float*>(ws),
                        reinterpret_cast<float2*>(w + part_bytes(a, D, splits)),
                        reinterpret_cast<int*>(w + part_bytes(a, D, splits) + ml_bytes(a, splits))};
    {
        TimedLaunch tl("paged_prefill", s);
        const dim3 grid((unsigned)most_items(a), splits);
        prefill_kernel<D, E4M3><<<grid, kThreads, Plan<D>::SMEM, s>>>(mq, mk, mv, mo, a, TB,
                                                                      hf ? 1 : 0, part);
        const kda_status st = launch_status();
        if (st != KDA_OK || splits == 1) return st;
    }
    TimedLaunch tl("paged_prefill_join", s);
    join_kernel<D><<<(unsigned)(((long long)a.T * a.HQ + 7) / 8), 256, 0, s>>>(a, part, splits);
    return launch_status();
}

}  // namespace

size_t paged_prefill_ws_bytes(const PagedArgs& a, int D, bool) {
    const int splits = most_splits(a);
    if (splits == 1) return 0;
    return part_bytes(a, D, splits) + ml_bytes(a, splits) + align256(sizeof(int));
}

kda_status paged_prefill_launch(const PagedArgs& a, int D, bool e4m3, void* ws, cudaStream_t s) {
    if (D == 128) return e4m3 ? launch<128, true>(a, ws, s) : launch<128, false>(a, ws, s);
    return e4m3 ? launch<64, true>(a, ws, s) : launch<64, false>(a, ws, s);
}

int* paged_prefill_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_prefill_error) == cudaSuccess ? static_cast<int*>(p)
                                                                         : nullptr;
}

}  // namespace kda
