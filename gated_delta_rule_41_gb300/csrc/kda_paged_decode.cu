// Attention of one new token per sequence over a paged key-value cache.
//
// For a key head and its G query heads the work is one pass over the visible
// rows of K and V: 4 G flop for each element read, so HBM bounds it (G = 4,
// bf16: 8 flop a byte) as long as the products run on the tensor cores.  The
// plan is therefore about keeping loads in flight and all SMs equally busy:
//
// * Work is cut into tiles of 64 tokens of one (sequence, key head, block of
//   query heads).  The tiles of all of them form one line, of which each
//   resident CTA takes an equal stretch (a prefix sum over the lengths, taken
//   by every CTA for itself), so a few long rows spread over the SMs like many
//   unequal ones.  A row that ends up in one CTA is written at once; of the
//   others each CTA leaves its part (sums, weights' maximum and total), and the
//   CTA that arrives last joins the parts in their order along the row, so the
//   result does not depend on which one that is.
// * A warp owns 16 tokens of a tile at a time.  They lie in one page (pages are
//   multiples of 16), so one table entry, read an iteration ahead, gives their
//   addresses.  K and V rows come by 16-byte asynchronous copies into the warp's own ring of stages;
//   no barrier is needed within a row.  Rows that the query does not see are
//   filled with zeros instead of being read.
// * S^T = K Q^T has the tokens on the M axis of mma.m16n8k16 and 8 query heads
//   on N, O^T = V^T P the channels on M, so up to 8 heads cost 16 MMAs for 16
//   tokens.  The transposed weights come from movmatrix.
// * Softmax: a running maximum m per head and warp, raised (and the sums
//   rescaled) only when a logit exceeds it by more than 2^8 in weight; the sums
//   are fp32, and weights up to 256 lose nothing in floating point.  Beside
//   e4m3 codes, which are exact in fp16, the weights enter the product with V
//   in fp16 (2^-11); beside bf16 values in two bf16 terms (2^-16), since one
//   alone (2^-8) would cost as much as the output's own rounding and the
//   second product is free here.
#include "kda_paged.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_paged_decode_error = 0;   // a kda_status

namespace {

using namespace paged;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGroup = 16;                 // tokens of a warp's step
constexpr int kPartHeads = 16;             // query heads of a CTA, at most

__device__ __forceinline__ void record() { atomicCAS(&g_paged_decode_error, 0, (int)KDA_ERR_SHAPE); }

// The visible tokens of a query as groups of 16: those of the sinks, then
// those from the window's start on.
struct Span {
    int len, low, sinks;     // token j is seen iff j < len and (j >= low or j < sinks)
    int nsink, first, n;     // groups of sinks; first group of the window; groups in all
    __device__ __forceinline__ int group(int i) const { return i < nsink ? i : i - nsink + first; }
    __device__ __forceinline__ int tiles() const { return max(1, (n + kWarps - 1) / kWarps); }
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
    // ring of stages: 24 KB (bf16, D = 128) per warp, two CTAs on an SM
    static constexpr int STAGES = RB == 256 ? 3 : RB == 128 ? 6 : 8;
    static constexpr int RING = STAGES * 2 * TILE;       // bytes per warp
    static constexpr int OS = D + 4;                     // row of the join buffer, floats
    static constexpr size_t SMEM = kWarps * RING;
    static_assert(NH * 8 * OS * 4 <= RING, "join buffer does not fit the ring");
};

// A part of a row: per head the maximum, the sum and D sums of a CTA.
template <int D>
struct Part {
    float m[kPartHeads], l[kPartHeads];
    float o[kPartHeads][D];
};

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kThreads, 2)
decode_kernel(const PagedArgs a, int HB, unsigned* __restrict__ tickets,
              Part<D>* __restrict__ parts) {
    using Sh = Shape<D, E4M3, NH>;
    constexpr int KS = D / 16;                           // k steps of S, m tiles of O
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_scan[kWarps];
    __shared__ int s_seq;
    __shared__ long long s_at;
    __shared__ float s_m[kWarps][kPartHeads], s_l[kWarps][kPartHeads];
    __shared__ unsigned s_ticket;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rows = a.HKV * HB;                         // rows of a sequence

    // ---- this CTA's stretch of the line of tiles ----
    const int per_thread = (a.S + kThreads - 1) / kThreads;
    const int s_lo = min(a.S, tid * per_thread), s_hi = min(a.S, s_lo + per_thread);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) mine += make_span(a, seq_len(a, s)).tiles();
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) s_scan[warp] = sum;
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
        for (;; ++s) {
            const long long n = (long long)make_span(a, seq_len(a, s)).tiles() * rows;
            if (begin < at + n) break;
            at += n;
        }
        s_seq = s;
        s_at = at;
    }
    __syncthreads();
    int s = s_seq;
    long long seq_at = s_at;                             // line index of sequence s's first tile
    const uint32_t ring = ptx::smem_u32(smem) + warp * Sh::RING;
    float* join = reinterpret_cast<float*>(smem + warp * Sh::RING);

    for (long long at = begin; at < end;) {
        Span sp = make_span(a, seq_len(a, s));
        while (at >= seq_at + (long long)sp.tiles() * rows) {
            seq_at += (long long)sp.tiles() * rows;
            sp = make_span(a, seq_len(a, ++s));
        }
        const int tiles = sp.tiles();
        const int row = (int)((at - seq_at) / tiles), tile0 = (int)((at - seq_at) % tiles);
        const int tile1 = (int)min((long long)tiles, tile0 + (end - at));
        const int h = row / HB, hq0 = h * a.G + row % HB * (8 * NH);
        const int heads = min(8 * NH, (h + 1) * a.G - hq0);

        // ---- Q as the B operand: head g (+ 8 n), channels of this lane ----
        // e4m3: q in fp16, scaled by a power of two to at most 2 (put back into
        // the logits' factor); channel pairs in the order that a 32-bit piece
        // of a K row gives them.
        uint32_t qf[NH][KS][2];
        float f[NH][2];                                  // logit factors of heads 2t, 2t + 1
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const bool on = 8 * n + g < heads;
            const __nv_bfloat16* q = a.q + s * a.q_stride + (long long)(hq0 + 8 * n + g) * D;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (E4M3) {
                    const uint2 x = on ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * t)
                                       : make_uint2(0, 0);
                    qf[n][k][0] = x.x;
                    qf[n][k][1] = x.y;
                } else {
                    qf[n][k][0] = on ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t) : 0;
                    qf[n][k][1] = on ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t + 8) : 0;
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
                // exponent of the largest, as far as 2^-e is a normal number
                const int e = max(-126, min(126, (int)(__float_as_uint(top) >> 23) - 127));
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

        // ---- the warp's groups of this stretch: gi0, gi0 + 4, ... ----
        const int gi0 = tile0 * kWarps + warp, gi1 = min(sp.n, tile1 * kWarps);
        const int steps = gi0 < gi1 ? (gi1 - gi0 + kWarps - 1) / kWarps : 0;
        const int* table = a.table + (size_t)s * a.max_pages;
        const int gshift = a.page_shift - 4;             // groups per page, log2
        auto page_of = [&](int i) {
            return i < steps ? __ldg(table + (sp.group(gi0 + i * kWarps) >> gshift)) : 0;
        };
        auto issue = [&](int i, int page) {
            if (i < steps) {
                const int grp = sp.group(gi0 + i * kWarps), j0 = grp * kGroup;
                const bool good = (unsigned)page < (unsigned)a.num_pages;
                if (!good) record();
                const long long off = (good ? page : 0) * a.page_stride +
                                      (grp & ((1 << gshift) - 1)) * kGroup * a.token_stride +
                                      h * a.head_stride;
                const char* kp = static_cast<const char*>(a.kp) + off * (E4M3 ? 1 : 2);
                const char* vp = static_cast<const char*>(a.vp) + off * (E4M3 ? 1 : 2);
                const long long ts = a.token_stride * (E4M3 ? 1 : 2);
                const uint32_t st = ring + (i % Sh::STAGES) * (2 * Sh::TILE);
#pragma unroll
                for (int r = 0; r < Sh::TILE / 512; ++r) {
                    const int x = r * 32 + lane, row_ = x / Sh::RC, c = x % Sh::RC;
                    const int j = j0 + row_;
                    const bool on = good && j < sp.len && (j >= sp.low || j < sp.sinks);
                    // chunks are permuted within 128 bytes so that eight rows of
                    // one chunk lie in different banks
                    const int sw = Sh::RC >= 8 ? (row_ & 7) : ((row_ >> 1) & 3);
                    const uint32_t d = st + row_ * Sh::RB + ((c ^ sw) << 4);
                    const long long o = row_ * ts + c * 16;
                    cp_async16_zfill(d, kp + o, on);
                    cp_async16_zfill(d + Sh::TILE, vp + o, on);
                }
            }
            ptx::cp_async_commit();
        };
        int page = page_of(0);
#pragma unroll
        for (int i = 0; i < Sh::STAGES - 1; ++i) {
            const int next = page_of(i + 1);
            issue(i, page);
            page = next;
        }

        float o[NH][KS][4], m[NH][2], l[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][k][i] = 0.f;
        }

        for (int i = 0; i < steps; ++i) {
            const int next = page_of(i + Sh::STAGES);
            cp_async_wait<Sh::STAGES - 2>();
            __syncwarp();                                // every lane's copies, and step i - 1 read
            issue(i + Sh::STAGES - 1, page);
            page = next;
            const uint32_t kt = ring + (i % Sh::STAGES) * (2 * Sh::TILE), vt = kt + Sh::TILE;

            // ---- S^T = K Q^T ----
            float x[NH][4];
#pragma unroll
            for (int n = 0; n < NH; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
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
                            mma16816<false>(x[n], af, qf[n][k][0], qf[n][k][1]);
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
                                mma16816<true>(x[n], af, qf[n][k + e][0], qf[n][k + e][1]);
                        }
                    }
                }
            }

            // ---- weights ----
            const int j0 = sp.group(gi0 + i * kWarps) * kGroup;
            const bool edge = j0 + kGroup > sp.len || (j0 < sp.low);
            bool rise = false;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[n][e] *= f[n][e & 1];
                    if (edge) {
                        const int j = j0 + g + 8 * (e >> 1);
                        if (!(j < sp.len && (j >= sp.low || j < sp.sinks))) x[n][e] = -INFINITY;
                    }
                    rise |= x[n][e] > m[n][e & 1] + 8.f;
                }
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(m[n][c], fmaxf(x[n][c], x[n][c + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float keep = m[n][c] == top ? 1.f : ex2(m[n][c] - top);
                        m[n][c] = top;
                        l[n][c] *= keep;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[n][k][c] *= keep;
                            o[n][k][c + 2] *= keep;
                        }
                    }
            }
            uint32_t pf[NH][2], pl[NH][2];               // weights (bf16: and what they lost)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float top = m[n][e & 1];
                    w[e] = ex2(x[n][e] - (top == -INFINITY ? 0.f : top));
                }
                l[n][0] += w[0] + w[2];
                l[n][1] += w[1] + w[3];
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
                        mma16816<false>(o[n][k], af, pf[n][0], pf[n][1]);
                        mma16816<false>(o[n][k], af, pl[n][0], pl[n][1]);
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
                            mma16816<true>(o[n][k + e], af, pf[n][0], pf[n][1]);
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- join the warps ----
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
                const int head = 8 * n + 2 * t + c;
                if (g == 0) {
                    s_m[warp][head] = m[n][c];
                    s_l[warp][head] = l[n][c];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    // rows g, g + 8 of the m tile are channels g, g + 8 (bf16) or
                    // 2g, 2g + 1 (e4m3)
                    const int d0 = 16 * k + (E4M3 ? 2 * g : g);
                    join[head * Sh::OS + d0] = o[n][k][c];
                    join[head * Sh::OS + d0 + (E4M3 ? 1 : 8)] = o[n][k][c + 2];
                }
            }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        const float vs = E4M3 && a.vs ? a.vs[h] : 1.f;
        const long long row_at = seq_at + (long long)row * tiles;   // line index of the row
        Part<D>* part = parts + 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
        for (int i = tid; i < heads * (D / 4); i += kThreads) {
            const int head = i / (D / 4), d = i % (D / 4) * 4;
            float top = -INFINITY, sum_l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][head]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float k = s_m[w][head] == -INFINITY ? 0.f : ex2(s_m[w][head] - top);
                const float4 y = *reinterpret_cast<const float4*>(
                    smem + w * Sh::RING + (head * Sh::OS + d) * 4);
                sum_l += k * s_l[w][head];
                v.x += k * y.x;
                v.y += k * y.y;
                v.z += k * y.z;
                v.w += k * y.w;
            }
            if (whole) {
                const float inv = top == -INFINITY ? 0.f : vs / sum_l;
                const long long out = (long long)s * a.HQ + hq0 + head;
                *reinterpret_cast<uint2*>(a.o + out * D + d) = make_uint2(
                    ptx::pack_bf16(v.x * inv, v.y * inv), ptx::pack_bf16(v.z * inv, v.w * inv));
                if (a.lse && d == 0)
                    a.lse[out] = top == -INFINITY ? -INFINITY : (top + lg2(sum_l)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(&part->o[head][d]) = v;
                if (d == 0) {
                    part->m[head] = top;
                    part->l[head] = sum_l;
                }
            }
        }
        if (!whole) {
            // ---- the row's parts: CTA c0 holds its first tile, c1 its last ----
            const int c0 = (int)(row_at / per), c1 = (int)((row_at + tiles - 1) / per);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_ticket = atomicAdd(tickets + c0, 1u);
            __syncthreads();
            if (s_ticket == (unsigned)(c1 - c0)) {
                __threadfence();
                if (tid == 0) tickets[c0] = 0;           // as the next call expects it
                for (int i = tid; i < heads * (D / 4); i += kThreads) {
                    const int head = i / (D / 4), d = i % (D / 4) * 4;
                    float top = -INFINITY, sum_l = 0.f;
                    for (int c = c0; c <= c1; ++c)
                        top = fmaxf(top, __ldcg(&parts[2 * c + (c == c0)].m[head]));
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const Part<D>* p = parts + 2 * c + (c == c0);
                        const float pm = __ldcg(&p->m[head]);
                        const float k = pm == -INFINITY ? 0.f : ex2(pm - top);
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(&p->o[head][d]));
                        sum_l += k * __ldcg(&p->l[head]);
                        v.x += k * y.x;
                        v.y += k * y.y;
                        v.z += k * y.z;
                        v.w += k * y.w;
                    }
                    const float inv = top == -INFINITY ? 0.f : vs / sum_l;
                    const long long out = (long long)s * a.HQ + hq0 + head;
                    *reinterpret_cast<uint2*>(a.o + out * D + d) = make_uint2(
                        ptx::pack_bf16(v.x * inv, v.y * inv), ptx::pack_bf16(v.z * inv, v.w * inv));
                    if (a.lse && d == 0)
                        a.lse[out] = top == -INFINITY ? -INFINITY : (top + lg2(sum_l)) * kLn2;
                }
            }
        }
        __syncthreads();                                 // the join buffers are read
        at += tile1 - tile0;
    }
}

// CTAs of a call: two on each SM.  The workspace does not depend on lengths.
int decode_grid() { return 2 * sm_count(); }

template <int D, bool E4M3, int NH>
kda_status launch(const PagedArgs& a, void* ws, cudaStream_t s) {
    using Sh = Shape<D, E4M3, NH>;
    static bool set[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_CUDA;
    auto* fn = decode_kernel<D, E4M3, NH>;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Sh::SMEM) != cudaSuccess)
            return KDA_ERR_CUDA;
        set[dev] = true;
    }
    const int HB = (a.G + 8 * NH - 1) / (8 * NH), W = decode_grid();
    const long long most = (long long)a.S * a.HKV * HB * ((a.cap + 63LL) / 64 + 1);
    TimedLaunch tl("paged_decode", s);
    fn<<<(unsigned)(most < W ? most : W), kThreads, Sh::SMEM, s>>>(
        a, HB, static_cast<unsigned*>(ws),
        reinterpret_cast<Part<D>*>(static_cast<char*>(ws) + align256(W * sizeof(unsigned))));
    return launch_status();
}

}  // namespace

size_t paged_decode_ws_bytes(const PagedArgs&, int D, bool) {
    const size_t W = decode_grid();
    return align256(W * sizeof(unsigned)) +
           align256(2 * W * (D == 128 ? sizeof(Part<128>) : sizeof(Part<64>)));
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

kda_status paged_decode_take_error(cudaStream_t s) {
    int err = 0;
    if (cudaMemcpyFromSymbolAsync(&err, g_paged_decode_error, sizeof(int), 0,
                                  cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return KDA_ERR_CUDA;
    if (err == 0) return KDA_OK;
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_paged_decode_error, &zero, sizeof(int), 0,
                                cudaMemcpyHostToDevice, s) != cudaSuccess)
        return KDA_ERR_CUDA;
    cudaStreamSynchronize(s);
    return static_cast<kda_status>(err);
}

}  // namespace kda
