// Page bookkeeping of the paged key-value cache: fork, extend, free, compact
// and the page copies behind them.  Everything runs on the device in stream
// order, so that a serving loop learns no length on the host.
//
// The plans (which free page goes to which request; which held page moves into
// which hole) are prefix sums over the requests and the pages' counts, taken
// by one CTA, 16384 counts a round; a plan takes about 2 us up to that many
// pages, and bounds a call of few pages.  The copies run over all SMs and are
// bounded by HBM: 128 forks of 786 KB (12 pools) take 17 us with their plan, 6
// TB/s; 515 moves of 262 KB (4 pools) 45 us.
#include <algorithm>

#include "kda_paged.cuh"
#include "kda_timing.cuh"

namespace kda {

__device__ int g_pages_error = 0;   // a kda_status

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPages = 16;      // counts of a thread at a time
constexpr int kCopyThreads = 256;

__device__ __forceinline__ void record(kda_status code) { atomicCAS(&g_pages_error, 0, code); }

// Workspace: the plan of one call.
struct Plan {
    int* count;    // [1] pairs in src, dst
    int* before;   // [S + 1] pages wanted before request i
    int* first;    // [S] extend: table column of request i's first new page; fork: its length
    int* src;      // [num_pages] page copies (fork: [n <= S])
    int* dst;
    int* rank;     // [num_pages] index of a moving page among the moving ones; or free pages
};

size_t plan_ints(const kda_pages_dims& d) {
    return 64 + 2 * ((size_t)d.S + 64) + 2 * (size_t)std::max(d.num_pages, d.S) + d.num_pages;
}

Plan carve(const kda_pages_dims& d, void* ws) {
    const size_t m = std::max(d.num_pages, d.S);
    Plan p;
    p.count = static_cast<int*>(ws);
    p.before = p.count + 64;
    p.first = p.before + d.S + 64;
    p.src = p.first + d.S + 64;
    p.dst = p.src + m;
    p.rank = p.dst + m;
    return p;
}

// Exclusive prefix sum of one value per thread over the CTA; *total: the sum.
// s: 32 values of scratch; the barriers order its use by successive calls.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T w = s[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s[lane] = w;
    }
    __syncthreads();
    const T base = warp ? s[warp - 1] : 0;
    *total = s[31];
    __syncthreads();
    return base + x - v;
}

// before[i] for the threads' requests in turn; sums past num_pages, which no
// pool can serve, are held at num_pages + 1.
__device__ __forceinline__ void scan_wants(long long* run, int want, int i, int n, int num_pages,
                                           long long* s, int* before) {
    long long total;
    const long long b = *run + block_scan<long long>(want, s, &total);
    const long long most = (long long)num_pages + 1;
    if (i < n) before[i] = (int)(b < most ? b : most);
    *run += total;
    if (threadIdx.x == 0) before[n] = (int)(*run < most ? *run : most);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size != 0);
}

// Counts of pages [p0, p0 + 16); past the end: -1.
__device__ __forceinline__ void load_counts(const int* refs, int num_pages, int p0,
                                            int (&r)[kPlanPages]) {
    if ((reinterpret_cast<uintptr_t>(refs) & 15) == 0 && p0 + kPlanPages <= num_pages) {
#pragma unroll
        for (int i = 0; i < kPlanPages; i += 4) {
            const int4 x = *reinterpret_cast<const int4*>(refs + p0 + i);
            r[i] = x.x;
            r[i + 1] = x.y;
            r[i + 2] = x.z;
            r[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPlanPages; ++i) r[i] = p0 + i < num_pages ? refs[p0 + i] : -1;
    }
}

// Lists the lowest free pages, in order, `wanted` of them or all; returns how
// many there are.
__device__ int list_free(int num_pages, const int* refs, int wanted, int* list, int* s) {
    int found = 0;
    for (int at = 0; at < num_pages && found < wanted; at += kPlanThreads * kPlanPages) {
        const int p0 = at + threadIdx.x * kPlanPages;
        int count[kPlanPages], mine = 0;
        load_counts(refs, num_pages, p0, count);
#pragma unroll
        for (int i = 0; i < kPlanPages; ++i) mine += count[i] == 0;
        int total;
        int r = found + block_scan<int>(mine, s, &total);
#pragma unroll
        for (int i = 0; i < kPlanPages; ++i)
            if (count[i] == 0) {
                if (r < wanted) list[r] = p0 + i;
                ++r;
            }
        found += total;
    }
    __syncthreads();
    return min(found, wanted);
}

// Deals listed pages out: request i takes before[i + 1] - before[i] of them, in
// order.  `take(i, k, page)` stores the k-th page of request i.
template <typename F>
__device__ void deal(const int* list, int found, const int* before, int n, F take) {
    for (int r = threadIdx.x; r < found; r += kPlanThreads) {
        int lo = 0, hi = n;   // the last request with before <= r: one that wants pages
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= r) lo = mid;
            else hi = mid;
        }
        take(lo, r - before[lo], list[r]);
    }
}

// ---- extend ----
// One CTA.  Request i wants the pages that row i's new length needs beyond
// those it holds; those that the listed free pages do not cover are refused as
// a whole, and their rows stay as they were.  `granted` (may be null): the
// tokens that each row gained.
__global__ void __launch_bounds__(kPlanThreads)
extend_kernel(kda_pages_dims d, const int* __restrict__ add, int add_all, int* table, int* lens,
              int* refs, int* granted, Plan pl) {
    __shared__ long long s_wide[32];
    __shared__ int s[32];
    const long long cap = (long long)d.max_pages * d.page_size;
    // tokens that row i gains, -1 if it cannot
    auto gain = [&](int i, int len) {
        const int more = add ? add[i] : (len > 0 ? add_all : 0);
        return len < 0 || more < 0 || (long long)len + more > cap ? -1 : more;
    };
    long long run = 0;
    for (int at = 0; at < d.S; at += kPlanThreads) {
        const int i = at + threadIdx.x;
        int want = 0;
        if (i < d.S) {
            const int len = lens[i], more = gain(i, len);
            if (more < 0) {
                record(KDA_ERR_SHAPE);
            } else {
                pl.first[i] = pages_of(len, d.page_size);
                want = pages_of(len + more, d.page_size) - pl.first[i];
            }
        }
        scan_wants(&run, want, i, d.S, d.num_pages, s_wide, pl.before);
    }
    __syncthreads();
    const int have = list_free(d.num_pages, refs, pl.before[d.S], pl.rank, s);
    deal(pl.rank, have, pl.before, d.S, [&](int i, int k, int page) {
        if (pl.before[i + 1] > have) return;
        table[(size_t)i * d.max_pages + pl.first[i] + k] = page;
        refs[page] = 1;
    });
    for (int i = threadIdx.x; i < d.S; i += kPlanThreads) {
        const int len = lens[i], more = gain(i, len);
        if (granted) granted[i] = 0;
        if (more <= 0) continue;
        if (pages_of(len + more, d.page_size) > pages_of(len, d.page_size) &&
            pl.before[i + 1] > have) {
            record(KDA_ERR_PAGES);
            continue;
        }
        lens[i] = len + more;
        if (granted) granted[i] = more;
    }
}

// ---- fork ----
// One CTA: request i wants a page if its parent's last page is partial.
// Leaves the copies (src, dst; -1 where there is none) and the lengths
// (first), and marks refused requests with src = -2.
__global__ void __launch_bounds__(kPlanThreads)
fork_plan_kernel(kda_pages_dims d, const int* __restrict__ parents,
                 const int* __restrict__ children, int n, const int* __restrict__ table,
                 const int* __restrict__ lens, int* refs, Plan pl) {
    __shared__ long long s_wide[32];
    __shared__ int s[32];
    paged::let_next_start();
    long long run = 0;
    for (int at = 0; at < n; at += kPlanThreads) {
        const int i = at + threadIdx.x;
        int want = 0;
        if (i < n) {
            const int p = parents[i], c = children[i];
            int src = -2;
            if ((unsigned)p < (unsigned)d.S && (unsigned)c < (unsigned)d.S && lens[c] == 0) {
                const int len = lens[p];
                if (len >= 0 && (long long)len <= (long long)d.max_pages * d.page_size) {
                    src = -1;
                    pl.first[i] = len;
                    if (len % d.page_size != 0) {
                        src = table[(size_t)p * d.max_pages + len / d.page_size];
                        want = 1;
                        if ((unsigned)src >= (unsigned)d.num_pages) {
                            src = -2;
                            want = 0;
                        }
                    }
                }
            }
            if (src == -2) record(KDA_ERR_SHAPE);
            pl.src[i] = src;
            pl.dst[i] = -1;
        }
        scan_wants(&run, want, i, n, d.num_pages, s_wide, pl.before);
    }
    __syncthreads();
    const int have = list_free(d.num_pages, refs, pl.before[n], pl.rank, s);
    deal(pl.rank, have, pl.before, n, [&](int i, int, int page) {
        pl.dst[i] = page;
        refs[page] = 1;
    });
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (pl.src[i] >= 0 && pl.dst[i] < 0) {
            record(KDA_ERR_PAGES);
            pl.src[i] = -2;
        }
}

struct Pools {
    kda_page_pool p[KDA_MAX_POOLS];
    int n;
};

// Copies piece `piece` of page src of a pool to page dst.  A CTA moves
// kPieceBytes: each thread has eight 16-byte loads in flight.
constexpr int kPieceBytes = kCopyThreads * 16 * 8;

__device__ __forceinline__ void copy_piece(const kda_page_pool& pool, long long src, long long dst,
                                           long long piece) {
    const long long o = piece * kPieceBytes;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(pool.base) +
                                                       src * pool.page_stride_bytes + o);
    uint4* to = reinterpret_cast<uint4*>(static_cast<char*>(pool.base) +
                                         dst * pool.page_stride_bytes + o);
    const long long left = (pool.page_bytes - o) / 16;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = threadIdx.x + i * kCopyThreads;
        if (j < left) x[i] = __ldcs(from + j);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = threadIdx.x + i * kCopyThreads;
        if (j < left) __stcs(to + j, x[i]);
    }
}

// Page copies (src[r], dst[r]), r < n (or *count).  blockIdx.y = pool; the
// CTAs of a row share the pool's (pair, piece) items.
__device__ __forceinline__ void copy_pages(const Pools& pools, int num_pages,
                                           const int* __restrict__ src,
                                           const int* __restrict__ dst, int n) {
    const kda_page_pool& pool = pools.p[blockIdx.y];
    const long long pieces = (pool.page_bytes + kPieceBytes - 1) / kPieceBytes;
    for (long long it = blockIdx.x; it < pieces * n; it += gridDim.x) {
        const int r = (int)(it / pieces);
        const int a = src[r], b = dst[r];
        if (a < 0 || b < 0) continue;
        if (a >= num_pages || b >= num_pages) {
            if (threadIdx.x == 0) record(KDA_ERR_SHAPE);
            continue;
        }
        copy_piece(pool, a, b, it % pieces);
    }
}

__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(const __grid_constant__ Pools pools, int num_pages, const int* __restrict__ src,
            const int* __restrict__ dst, int n) {
    copy_pages(pools, num_pages, src, dst, n);
}

// blockIdx.y == number of pools: the children's rows, one per CTA in turn;
// else the page copies.
__global__ void __launch_bounds__(kCopyThreads)
fork_kernel(const __grid_constant__ Pools pools, kda_pages_dims d,
            const int* __restrict__ parents, const int* __restrict__ children, int n, int* table,
            int* lens, int* refs, Plan pl) {
    paged::wait_for_previous();
    if ((int)blockIdx.y < pools.n) {
        copy_pages(pools, d.num_pages, pl.src, pl.dst, n);
        return;
    }
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
        const int src = pl.src[i];
        if (src == -2) continue;
        const int p = parents[i], c = children[i];
        const int len = pl.first[i], full = len / d.page_size;
        const int* from = table + (size_t)p * d.max_pages;
        int* to = table + (size_t)c * d.max_pages;
        for (int j = threadIdx.x; j < d.max_pages; j += kCopyThreads) {
            int page = -1;
            if (j < full) {
                page = from[j];
                if ((unsigned)page < (unsigned)d.num_pages) atomicAdd(refs + page, 1);
                else record(KDA_ERR_SHAPE);
            } else if (j == full && src >= 0) {
                page = pl.dst[i];
            }
            to[j] = page;
        }
        if (threadIdx.x == 0) lens[c] = len;
    }
}

// ---- free ----
__global__ void __launch_bounds__(kCopyThreads)
free_kernel(kda_pages_dims d, const int* __restrict__ slots, int* table, int* lens, int* refs) {
    const int row = slots[blockIdx.x];
    if ((unsigned)row >= (unsigned)d.S) {
        if (threadIdx.x == 0) record(KDA_ERR_SHAPE);
        return;
    }
    int* t = table + (size_t)row * d.max_pages;
    for (int j = threadIdx.x; j < d.max_pages; j += kCopyThreads) {
        const int page = t[j];
        if (page < 0) continue;
        t[j] = -1;
        if (page >= d.num_pages) {
            record(KDA_ERR_SHAPE);
        } else if (atomicSub(refs + page, 1) <= 0) {
            atomicAdd(refs + page, 1);
            record(KDA_ERR_SHAPE);
        }
    }
    if (threadIdx.x == 0) lens[row] = 0;
}

// ---- compact ----
// One CTA: L = the number of held pages; the held pages at or above L (src,
// with their rank) and the others below L (dst), each in rising order; the
// two lists are equally long, since every page is one or the other: a negative
// count, which no book keeps, is reported and not held.  Then the counts move
// along.
__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(int num_pages, int* refs, Plan pl) {
    __shared__ long long s[32];
    paged::let_next_start();
    long long total, L = 0;
    for (int p0 = threadIdx.x * kPlanPages; p0 < num_pages; p0 += kPlanThreads * kPlanPages) {
        int count[kPlanPages];
        load_counts(refs, num_pages, p0, count);
#pragma unroll
        for (int i = 0; i < kPlanPages; ++i) {
            L += count[i] > 0;
            if (count[i] < 0 && p0 + i < num_pages) record(KDA_ERR_SHAPE);
        }
    }
    block_scan<long long>(L, s, &total);
    L = total;
    // holes and moves before this thread's pages, in the halves of one sum
    long long run = 0;
    for (int at = 0; at < num_pages; at += kPlanThreads * kPlanPages) {
        const int p0 = at + threadIdx.x * kPlanPages;
        int count[kPlanPages];
        load_counts(refs, num_pages, p0, count);
        long long mine = 0;
#pragma unroll
        for (int i = 0; i < kPlanPages; ++i) {
            if (count[i] <= 0 && p0 + i < L) ++mine;
            if (count[i] > 0 && p0 + i >= L) mine += 1LL << 32;
        }
        const long long before = run + block_scan<long long>(mine, s, &total);
        run += total;
        int h = (int)(before & 0xffffffff), m = (int)(before >> 32);
        if (mine != 0) {
#pragma unroll
            for (int i = 0; i < kPlanPages; ++i) {
                if (count[i] <= 0 && p0 + i < L) pl.dst[h++] = p0 + i;
                if (count[i] > 0 && p0 + i >= L) {
                    pl.src[m] = p0 + i;
                    pl.rank[p0 + i] = m++;
                }
            }
        }
    }
    const int moves = (int)(run >> 32);
    __syncthreads();
    for (int r = threadIdx.x; r < moves; r += kPlanThreads) {
        refs[pl.dst[r]] = refs[pl.src[r]];
        refs[pl.src[r]] = 0;
    }
    if (threadIdx.x == 0) {
        pl.count[0] = moves;
        pl.count[1] = (int)L;
    }
}

// blockIdx.y == number of pools: the table; else the page copies.
__global__ void __launch_bounds__(kCopyThreads)
compact_kernel(const __grid_constant__ Pools pools, kda_pages_dims d, int* table, Plan pl) {
    paged::wait_for_previous();
    const int moves = pl.count[0], L = pl.count[1];
    if ((int)blockIdx.y < pools.n) {
        copy_pages(pools, d.num_pages, pl.src, pl.dst, moves);
        return;
    }
    const long long n = (long long)d.S * d.max_pages;
    for (long long i = (long long)blockIdx.x * kCopyThreads + threadIdx.x; i < n;
         i += (long long)gridDim.x * kCopyThreads) {
        const int page = table[i];
        if (page < L) continue;
        if (page >= d.num_pages) {
            record(KDA_ERR_SHAPE);
            continue;
        }
        const int m = pl.rank[page];
        // a page that the table names though its count is zero did not move
        if ((unsigned)m < (unsigned)moves && pl.src[m] == page) table[i] = pl.dst[m];
        else record(KDA_ERR_SHAPE);
    }
}

Pools make_pools(const kda_page_pool* pools, int n) {
    Pools p = {};
    p.n = n;
    for (int i = 0; i < n; ++i) p.p[i] = pools[i];
    return p;
}

// CTAs per pool: enough to fill the SMs several times over, no more than the
// pairs have pieces.
int copy_grid(const kda_page_pool* pools, int num_pools, long long pairs) {
    long long most = 1;
    for (int i = 0; i < num_pools; ++i)
        most = std::max(most, (pools[i].page_bytes + kPieceBytes - 1) / kPieceBytes);
    const long long want = std::max(1, paged::sm_count() * 8 / std::max(1, num_pools));
    return (int)std::max<long long>(1, std::min(want, most * pairs));
}

}  // namespace

size_t pages_ws_bytes(const kda_pages_dims& d) { return align256(plan_ints(d) * sizeof(int)); }

kda_status pages_extend_launch(const kda_pages_dims& d, const int* add, int add_all, int* table,
                               int* lens, int* refs, int* granted, void* ws, cudaStream_t s) {
    TimedLaunch tl("pages_extend", s);
    extend_kernel<<<1, kPlanThreads, 0, s>>>(d, add, add_all, table, lens, refs, granted,
                                             carve(d, ws));
    return launch_status();
}

kda_status pages_fork_launch(const kda_pages_dims& d, const kda_page_pool* pools, int num_pools,
                             const int* parents, const int* children, int n, int* table,
                             int* lens, int* refs, void* ws, cudaStream_t s) {
    const Plan pl = carve(d, ws);
    {
        TimedLaunch tl("pages_fork_plan", s);
        fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(d, parents, children, n, table, lens, refs, pl);
        const kda_status st = launch_status();
        if (st != KDA_OK) return st;
    }
    TimedLaunch tl("pages_fork", s);
    const dim3 grid(std::max(copy_grid(pools, num_pools, n), std::min(n, paged::sm_count())),
                    num_pools + 1);
    return paged::launch_overlapped(fork_kernel, grid, kCopyThreads, 0, s,
                                    make_pools(pools, num_pools), d, parents, children, n, table,
                                    lens, refs, pl);
}

kda_status pages_free_launch(const kda_pages_dims& d, const int* slots, int n, int* table,
                             int* lens, int* refs, cudaStream_t s) {
    TimedLaunch tl("pages_free", s);
    free_kernel<<<n, kCopyThreads, 0, s>>>(d, slots, table, lens, refs);
    return launch_status();
}

kda_status pages_compact_launch(const kda_pages_dims& d, const kda_page_pool* pools,
                                int num_pools, int* table, int* refs, void* ws, cudaStream_t s) {
    const Plan pl = carve(d, ws);
    {
        TimedLaunch tl("pages_compact_plan", s);
        compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(d.num_pages, refs, pl);
        const kda_status st = launch_status();
        if (st != KDA_OK) return st;
    }
    TimedLaunch tl("pages_compact", s);
    const dim3 grid(copy_grid(pools, num_pools, d.num_pages), num_pools + 1);
    return paged::launch_overlapped(compact_kernel, grid, kCopyThreads, 0, s,
                                    make_pools(pools, num_pools), d, table, pl);
}

kda_status pages_copy_launch(const kda_page_pool* pools, int num_pools, int num_pages,
                             const int* src, const int* dst, int n, cudaStream_t s) {
    TimedLaunch tl("pages_copy", s);
    const dim3 grid(copy_grid(pools, num_pools, n), num_pools);
    copy_kernel<<<grid, kCopyThreads, 0, s>>>(make_pools(pools, num_pools), num_pages, src, dst,
                                              n);
    return launch_status();
}

int* pages_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_pages_error) == cudaSuccess ? static_cast<int*>(p) : nullptr;
}

}  // namespace kda
