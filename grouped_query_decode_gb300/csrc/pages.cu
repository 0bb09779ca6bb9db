// Page management of a paged cache: which page belongs to which sequence
// (block table, reference counts) and the copies of pages that follow from it.
//
// Every call is decided on the device, in one planning kernel, and carried out
// by a second kernel over the whole GPU that reads the plan from the
// workspace; the host never waits and a call can be captured into a graph. The
// planning kernel is one cluster of eight CTAs: what it reads once (counts of
// up to millions of pages) is shared by 256 warps, and what the warps need of
// each other (how many free pages lie before mine) goes through distributed
// shared memory in one exchange.
// What bounds it: the plan is latency (a cluster's start, one pass over the
// counts, one exchange, one pass over what it kept of them: 3 to 5 us up to 65536
// pages; one CTA took 13), the rest bytes. Measured: a fork of 32 beams, 1.3 MB of
// pages, 7.3 us; one of 64 beams over 64 layers, 167 MB, 31 us, 5.4 TB/s; 1 GB
// packed 163 us, 6.2 TB/s of 6.77 for a plain copy; pages reserved for 256
// sequences and given back in a pool of 65536, 11.1 us with three copies of the
// table, the lengths and the counts between the calls.
//
// All of it is integer work with one result: pages are taken in ascending
// order, ranks come from scans, and the only atomics add to integer counts.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_decode.h"
#include "gqa_launch.h"
#include "ptx.cuh"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;            // of a CTA
static_assert(kPlanWarps == 32, "a warp a lane");
constexpr int kAllWarps = kPlanCtas * kPlanWarps;
constexpr int kMoveThreads = 256;

// Workspace, in ints: the header, then the copies' source and destination
// pages (also the free pages of a reservation), then one number per row.
constexpr int kWsPairs = 0, kWsOk = 1, kWsLive = 2, kWsHeader = 64;
struct PageWs {
    int* head;
    int* src;       // [num_pages]
    int* dst;       // [num_pages]
    int* row_page;  // [B]
};
__host__ __device__ inline PageWs page_ws(void* ws, int num_pages) {
    int* p = static_cast<int*>(ws);
    return {p, p + kWsHeader, p + kWsHeader + num_pages, p + kWsHeader + 2 * (size_t)num_pages};
}

struct PoolSet {
    gqa_page_pool_t pool[GQA_MAX_POOLS];
    int n;
};

struct PagesParams {
    const int32_t* src_rows;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* refs;
    int32_t* table_out;
    int32_t* lens_out;
    int32_t* refs_out;
    int32_t* counts;
    void* ws;
    int B, max_pages, page_size, num_pages;
};

__device__ __forceinline__ bool is_page(int e, int num_pages) { return (unsigned)e < (unsigned)num_pages; }

__device__ __forceinline__ int tokens_of(const PagesParams& p, int b) {
    const long long most = (long long)p.max_pages * p.page_size;
    const int t = p.lens[b];
    return t < 0 ? 0 : (t > most ? (int)most : t);
}

__device__ __forceinline__ int pages_for(const PagesParams& p, int tokens) {
    return tokens / p.page_size + (tokens % p.page_size != 0);
}

// Exclusive sum of one value per thread of the CTA, and the total.
__device__ int block_exclusive_sum(int v, int* total) {
    __shared__ int warp_sum[kPlanWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    const int s = warp_sum[lane];
    *total = __reduce_add_sync(0xffffffffu, s);
    return __reduce_add_sync(0xffffffffu, lane < warp ? s : 0) + x - v;
}

// x = row * n + column, of 64-bit x; in 32 bits where they do (a third of the time).
struct Entry {
    int row, column;
};
__device__ __forceinline__ Entry entry_of(long long x, int n) {
    if (x >> 32) return {(int)(x / n), (int)(x % n)};
    const unsigned q = (unsigned)x / (unsigned)n;
    return {(int)q, (int)((unsigned)x - q * (unsigned)n)};
}

// The cluster's warps share the pages in contiguous, ascending ranges. live:
// pages with a count > 0 before this warp's range, and of all pages. Lane k
// keeps which of the range's k-th 32 pages are live, so that what follows the
// exchange need not read the counts again (one round trip to L2 per 32 pages).
struct Ranks {
    int lo, hi, live_before, live;
    unsigned mask;
};
// The live pages among the 32 from lo + 32 k on.
__device__ __forceinline__ unsigned live_mask(const int32_t* refs, const Ranks& r, int k) {
    if (k < 32) return __shfl_sync(0xffffffffu, r.mask, k);
    const int i = r.lo + 32 * k + (threadIdx.x & 31);
    return __ballot_sync(0xffffffffu, i < r.hi && refs[i] > 0);
}
// Every thread of the cluster, which has called announce_start(); synchronises it
// (and so orders its global writes).
__device__ __forceinline__ void announce_start() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ Ranks rank_pages(const int32_t* refs, int num_pages) {
    __shared__ int warp_live[kPlanWarps];
    __shared__ int cta_live[kPlanCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = cluster.block_rank();
    const int per = ((num_pages + kAllWarps - 1) / kAllWarps + 31) / 32 * 32;
    Ranks r;
    r.lo = (int)min((long long)num_pages, (long long)(cta * kPlanWarps + warp) * per);
    r.hi = min(num_pages, r.lo + per);
    int n = 0;
    r.mask = 0;
    for (int k0 = 0; r.lo + 32 * k0 < r.hi; k0 += 8) {
        int count[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = r.lo + 32 * (k0 + k) + lane;
            count[k] = i < r.hi ? refs[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const unsigned m = __ballot_sync(0xffffffffu, count[k] > 0);
            n += __popc(m);
            if (lane == k0 + k) r.mask = m;
        }
    }
    if (lane == 0) warp_live[warp] = n;
    __syncthreads();
    const int of_lane = warp_live[lane];
    const int mine = __reduce_add_sync(0xffffffffu, of_lane);
    int before = __reduce_add_sync(0xffffffffu, lane < warp ? of_lane : 0);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // all CTAs have started
    if (threadIdx.x < kPlanCtas) cluster.map_shared_rank(cta_live, threadIdx.x)[cta] = mine;
    cluster.sync();
    r.live = 0;
    for (int c = 0; c < kPlanCtas; ++c) {
        if (c < cta) before += cta_live[c];
        r.live += cta_live[c];
    }
    r.live_before = before;
    return r;
}

// Calls f(page, free pages before it) for the free pages of the warp's range,
// those with at least `limit` before them excepted.
template <class F>
__device__ void each_free(const int32_t* refs, const Ranks& r, int limit, F f) {
    const int lane = threadIdx.x & 31;
    int at = r.lo - r.live_before;
    for (int q = 0; r.lo + 32 * q < r.hi && at < limit; ++q) {
        const int i = r.lo + 32 * q + lane;
        const int here = min(32, r.hi - (r.lo + 32 * q));
        const unsigned m = ~live_mask(refs, r, q) & (0xffffffffu >> (32 - here));
        const int k = at + __popc(m & ((1u << lane) - 1));
        if ((m >> lane & 1) && k < limit) f(i, k);
        at += __popc(m);
    }
}

// ------------------------------------------------------------------ planning

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    reserve_kernel(const PagesParams p) {
    announce_start();
    pdl_launch_dependents();
    pdl_wait_primary();
    const PageWs ws = page_ws(p.ws, p.num_pages);
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31;
    const int gw = cluster.block_rank() * kPlanWarps + (threadIdx.x >> 5);
    __shared__ int want[GQA_MAX_PAGE_ROWS];   // missing pages of the rows before each
    // Lane k keeps the first missing entry of the warp's k-th row, and its pages.
    static_assert(GQA_MAX_PAGE_ROWS <= 32 * kAllWarps, "a row a lane");
    int first = 0, pages = 0;
    for (int b = gw, k = 0; b < p.B; b += kAllWarps, ++k) {
        const int n = pages_for(p, tokens_of(p, b));
        int missing = 0, at = n;
#pragma unroll 4
        for (int j = lane; j < n; j += 32)
            if (!is_page(p.table_out[(size_t)b * p.max_pages + j], p.num_pages)) {
                ++missing;
                at = min(at, j);
            }
        missing = __reduce_add_sync(0xffffffffu, missing);
        at = __reduce_min_sync(0xffffffffu, at);
        if (lane == k) first = at, pages = n;
        if (lane == 0) ws.row_page[b] = missing;
    }
    const Ranks r = rank_pages(p.refs_out, p.num_pages);
    int need = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const int v = b < p.B ? ws.row_page[b] : 0;
        int total;
        const int before = block_exclusive_sum(v, &total);
        if (b < p.B) want[b] = need + before;
        need += total;
    }
    const int free = p.num_pages - r.live;
    if (gw == 0 && lane == 0) {
        p.counts[0] = need;
        p.counts[1] = free;
    }
    if (need == 0 || need > free) return;    // the whole cluster
    each_free(p.refs_out, r, need, [&](int page, int k) { ws.src[k] = page; });
    cluster.sync();
    for (int b = gw, k = 0; b < p.B; b += kAllWarps, ++k) {
        const int n = __shfl_sync(0xffffffffu, pages, k), j1 = __shfl_sync(0xffffffffu, first, k);
        int at = want[b];
        const int end = b + 1 < p.B ? want[b + 1] : need;
        for (int j0 = j1; j0 < n && at < end; j0 += 32) {
            const int j = j0 + lane;
            int32_t* e = p.table_out + (size_t)b * p.max_pages + j;
            const bool mine = j < n && !is_page(*e, p.num_pages);
            const unsigned m = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                const int page = ws.src[at + __popc(m & ((1u << lane) - 1))];
                *e = page;
                p.refs_out[page] = 1;
            }
            at += __popc(m);
        }
    }
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(const PagesParams p) {
    announce_start();
    pdl_launch_dependents();
    pdl_wait_primary();
    const PageWs ws = page_ws(p.ws, p.num_pages);
    const bool writes = cg::this_cluster().block_rank() == 0;
    __shared__ int first[GQA_MAX_PAGE_ROWS];   // the lowest row that goes on from each row
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) first[b] = p.B;
    __syncthreads();
    for (int i = threadIdx.x; i < p.B; i += kPlanThreads) {
        const int s = p.src_rows[i];
        if (s >= 0 && s < p.B) atomicMin(&first[s], i);
    }
    const Ranks r = rank_pages(p.refs, p.num_pages);   // synchronises the CTA
    for (int i = r.lo + (threadIdx.x & 31); i < r.hi; i += 32) p.refs_out[i] = p.refs[i];
    // Every CTA counts the copies of all rows; the first one notes them.
    int need = 0;
    for (int i0 = 0; i0 < p.B; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int old = -1;
        bool is_first = false;
        if (i < p.B) {
            const int s = p.src_rows[i];
            if (s >= 0 && s < p.B) {
                is_first = first[s] == i;
                const int t = tokens_of(p, s);
                if (!is_first && t % p.page_size) old = p.table[(size_t)s * p.max_pages + t / p.page_size];
            }
        }
        const bool copies = is_page(old, p.num_pages);
        int total;
        const int k = need + block_exclusive_sum(copies ? 1 : 0, &total);
        if (i < p.B && writes) {
            // The first row of each sequence takes its row as it is: -2.
            // Another row's copy is pair k, whose new page the second kernel
            // looks up, or none: -1.
            ws.row_page[i] = is_first ? -2 : copies ? k : -1;
            if (copies && k < p.num_pages) ws.src[k] = old;
        }
        need += total;
    }
    const int free = p.num_pages - r.live;
    if (writes && threadIdx.x == 0) {
        p.counts[0] = need;
        p.counts[1] = free;
        ws.head[kWsPairs] = need <= free ? need : 0;
        ws.head[kWsOk] = need <= free;
    }
    // A free page's count may lie below 0; the second kernel counts its new holder
    // from 0. (The lane that copied the count above writes it again.)
    if (need <= free)
        each_free(p.refs, r, need, [&](int page, int k) {
            ws.dst[k] = page;
            p.refs_out[page] = 0;
        });
}

// With `live` live pages, the free pages below `live` and the live ones from
// there on are as many, and the k-th of the one takes the k-th of the other. A
// free page i has i - (live pages before it) free ones before it, so both
// lists follow from the one exchange; the moved pages are listed in descending
// order, since it is the live pages behind a page that a warp knows.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(const PagesParams p) {
    announce_start();
    pdl_launch_dependents();
    pdl_wait_primary();
    const PageWs ws = page_ws(p.ws, p.num_pages);
    const int lane = threadIdx.x & 31;
    const Ranks r = rank_pages(p.refs, p.num_pages);
    int at = r.live_before;
    for (int q = 0; r.lo + 32 * q < r.hi; ++q) {
        const int i = r.lo + 32 * q + lane;
        const unsigned m = live_mask(p.refs, r, q);
        const bool live = m >> lane & 1;
        const int before = at + __popc(m & ((1u << lane) - 1));
        if (i < r.hi && !live && i < r.live) ws.dst[i - before] = i;
        if (live && i >= r.live) ws.src[r.live - 1 - before] = i;
        // The page before the boundary knows how many lie behind it.
        if (i < r.hi && i == r.live - 1) {
            const int moved = r.live - before - (live ? 1 : 0);
            ws.head[kWsPairs] = moved;
            p.counts[0] = moved;
        }
        at += __popc(m);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.counts[1] = r.live;
        ws.head[kWsLive] = r.live;
        if (r.live == 0) ws.head[kWsPairs] = p.counts[0] = 0;
    }
}

// ------------------------------------------------------------ carrying it out

// One warp's copy of at most kPiece bytes; 16-byte pieces load all before they
// store, so that a warp has 4 KB under way.
constexpr size_t kPiece = 4096;
template <class T>
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, size_t bytes, int lane) {
    const int n = (int)(bytes / sizeof(T));
    const T* from = reinterpret_cast<const T*>(src);
    T* to = reinterpret_cast<T*>(dst);
    if constexpr (sizeof(T) == 16) {
        constexpr int kAtOnce = (int)(kPiece / 16 / 32);
        T v[kAtOnce];
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c)
            if (lane + 32 * c < n) v[c] = __ldcs(from + lane + 32 * c);
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c)
            if (lane + 32 * c < n) __stcs(to + lane + 32 * c, v[c]);
    } else {
        for (int i = lane; i < n; i += 32) to[i] = from[i];
    }
}

// Pages src[k] -> dst[k], k < n, of every layer of every pool; one warp takes
// one piece of a page at a time.
template <bool SRC_DESCENDING>
__device__ void copy_pages(const PoolSet& pools, const int* src, const int* dst, int n, int num_pages) {
    const int lane = threadIdx.x & 31;
    const long long warp = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
    for (int q = 0; q < pools.n; ++q) {
        const gqa_page_pool_t pool = pools.pool[q];
        const long long pieces = (long long)((pool.page_bytes + kPiece - 1) / kPiece);
        const long long items = pieces * pool.layers * n;
        for (long long it = warp; it < items; it += warps) {
            long long piece;
            int k, layer;
            if (items >> 32) {
                const long long rest = it / pieces;
                piece = it - rest * pieces;
                k = (int)(rest / pool.layers);
                layer = (int)(rest - (long long)k * pool.layers);
            } else {
                const unsigned rest = (unsigned)it / (unsigned)pieces;
                piece = (unsigned)it - rest * (unsigned)pieces;
                k = (int)(rest / (unsigned)pool.layers);
                layer = (int)(rest - (unsigned)k * (unsigned)pool.layers);
            }
            const int a = src[SRC_DESCENDING ? n - 1 - k : k], b = dst[k];
            if (!is_page(a, num_pages) || !is_page(b, num_pages)) continue;
            char* base = static_cast<char*>(pool.base) + (size_t)layer * pool.layer_bytes + piece * kPiece;
            const char* from = base + (size_t)a * pool.page_bytes;
            char* to = base + (size_t)b * pool.page_bytes;
            const size_t bytes = min(kPiece, pool.page_bytes - (size_t)piece * kPiece);
            const uintptr_t bits = reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to) | bytes;
            if ((bits & 15) == 0)
                copy_bytes<uint4>(to, from, bytes, lane);
            else if ((bits & 3) == 0)
                copy_bytes<unsigned>(to, from, bytes, lane);
            else
                copy_bytes<unsigned char>(to, from, bytes, lane);
        }
    }
}

__global__ void __launch_bounds__(kMoveThreads) copy_kernel(const __grid_constant__ PoolSet pools,
                                                            const int* src, const int* dst, int n,
                                                            int num_pages) {
    pdl_launch_dependents();
    pdl_wait_primary();
    copy_pages<false>(pools, src, dst, n, num_pages);
}

__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const __grid_constant__ PoolSet pools,
                                                            const PagesParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const PageWs ws = page_ws(p.ws, p.num_pages);
    const bool ok = ws.head[kWsOk] != 0;
    const long long entries = (long long)p.B * p.max_pages;
    for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < entries;
         x += (long long)gridDim.x * blockDim.x) {
        const Entry e = entry_of(x, p.max_pages);
        const int i = e.row, j = e.column;
        const int was = p.table[x];
        int now = was;
        if (ok) {
            const int s = p.src_rows[i];
            now = -1;
            if (s >= 0 && s < p.B) {
                const int t = tokens_of(p, s);
                const int mark = ws.row_page[i];
                if (mark == -2 || j < t / p.page_size)
                    now = p.table[(size_t)s * p.max_pages + j];
                else if (mark >= 0 && j == t / p.page_size)
                    now = ws.dst[mark];
            }
            if (now != was) {
                if (is_page(was, p.num_pages)) atomicAdd(&p.refs_out[was], -1);
                if (is_page(now, p.num_pages)) atomicAdd(&p.refs_out[now], 1);
            }
        }
        p.table_out[x] = now;
        if (j == 0) {
            const int s = p.src_rows[i];
            p.lens_out[i] = !ok ? p.lens[i] : (s >= 0 && s < p.B ? tokens_of(p, s) : 0);
        }
    }
    copy_pages<false>(pools, ws.src, ws.dst, ws.head[kWsPairs], p.num_pages);
}

__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ PoolSet pools,
                                                               const PagesParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const PageWs ws = page_ws(p.ws, p.num_pages);
    const int live = ws.head[kWsLive], pairs = ws.head[kWsPairs];
    const long long stride = (long long)gridDim.x * blockDim.x;
    const long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    for (long long x = t0; x < (long long)p.B * p.max_pages; x += stride) {
        int e = p.table[x];
        if (is_page(e, p.num_pages) && e >= live) {
            // The moved pages are listed in descending order. An entry whose
            // page has no reference is none of them and stays.
            int lo = 0, hi = pairs;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (ws.src[mid] > e) lo = mid + 1; else hi = mid;
            }
            if (lo < pairs && ws.src[lo] == e) e = ws.dst[pairs - 1 - lo];
        }
        p.table_out[x] = e;
    }
    // In place, the counts of a moved page's two ends belong to its own thread
    // alone; every other thread may rewrite what it read.
    for (long long k = t0; k < pairs; k += stride) {
        const int a = ws.src[pairs - 1 - k], b = ws.dst[k], n = p.refs[a];
        p.refs_out[b] = n;
        p.refs_out[a] = 0;
    }
    if (p.refs_out != p.refs) {
        for (long long i = t0; i < p.num_pages; i += stride) {
            const int n = p.refs[i];
            if ((n > 0) == (i < live)) p.refs_out[i] = n;
        }
    }
    copy_pages<true>(pools, ws.src, ws.dst, pairs, p.num_pages);
}

__global__ void __launch_bounds__(kMoveThreads) free_kernel(const uint8_t* done, const PagesParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const long long entries = (long long)p.B * p.max_pages;
    for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < entries;
         x += (long long)gridDim.x * blockDim.x) {
        const Entry at = entry_of(x, p.max_pages);
        if (!done[at.row]) continue;
        const int e = p.table_out[x];
        if (is_page(e, p.num_pages) && atomicAdd(&p.refs_out[e], -1) <= 0) atomicAdd(&p.refs_out[e], 1);
        p.table_out[x] = -1;
        if (at.column == 0) p.lens_out[at.row] = 0;
    }
}

// ---------------------------------------------------------------------- host

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <class... KArgs, class... Args>
int launch(void (*kernel)(KArgs...), unsigned grid, unsigned threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

int check_pools(const gqa_page_pool_t* pools, int num_pools, int num_pages, PoolSet* set) {
    if (num_pools < 0 || (num_pools > 0 && !pools)) return GQA_ERR_INVALID_ARG;
    if (num_pools > GQA_MAX_POOLS) return GQA_ERR_UNSUPPORTED;
    for (int i = 0; i < num_pools; ++i) {
        const gqa_page_pool_t& q = pools[i];
        if (!q.base || q.page_bytes == 0 || q.layers <= 0 ||
            (q.layers > 1 && q.layer_bytes / (size_t)num_pages < q.page_bytes))
            return GQA_ERR_INVALID_ARG;
        set->pool[i] = q;
    }
    set->n = num_pools;
    return GQA_OK;
}

int check_sizes(int B, int max_pages, int page_size, int num_pages) {
    if (B <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0) return GQA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size >= (1ll << 31) || num_pages > (1 << 30)) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

// Whether any two of n ranges of memory share a byte.
struct Range {
    const void* at;
    size_t bytes;
};
template <int N>
bool overlap(const Range (&r)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < i; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].at), b = reinterpret_cast<uintptr_t>(r[j].at);
            if (a < b + r[j].bytes && b < a + r[i].bytes) return true;
        }
    return false;
}

int check_ws(void* ws, size_t bytes, int B, int num_pages) {
    if (!ws || bytes < gqa_pages_workspace_bytes(B, num_pages) || (reinterpret_cast<uintptr_t>(ws) & 255u))
        return GQA_ERR_WORKSPACE;
    return GQA_OK;
}

// The grid of a kernel that looks at `entries` table entries and then copies up
// to n pages: a thread per entry and a warp per piece of a page, at most eight
// CTAs per SM.
unsigned move_grid(const PoolSet& set, long long n, long long entries, int sms) {
    long long warps = (entries + 31) / 32;
    for (int i = 0; i < set.n; ++i)
        warps += n * set.pool[i].layers * (long long)((set.pool[i].page_bytes + kPiece - 1) / kPiece);
    const long long most = (long long)sms * 8, want = (warps * 32 + kMoveThreads - 1) / kMoveThreads;
    return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_pages_workspace_bytes(int B, int num_pages) {
    if (B <= 0 || num_pages <= 0) return 0;
    return sizeof(int) * ((size_t)kWsHeader + 2 * (size_t)num_pages + (size_t)B);
}

int gqa_pages_copy(const gqa_page_pool_t* pools, int num_pools, const int32_t* src, const int32_t* dst, int n,
                   int num_pages, cudaStream_t stream) {
    if (n < 0 || num_pages <= 0) return GQA_ERR_INVALID_ARG;
    PoolSet set;
    int st = check_pools(pools, num_pools, num_pages, &set);
    if (st != GQA_OK) return st;
    if (n == 0 || num_pools == 0) return GQA_OK;
    if (!src || !dst) return GQA_ERR_INVALID_ARG;
    if (!aligned4(src) || !aligned4(dst)) return GQA_ERR_MISALIGNED;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    return launch(copy_kernel, move_grid(set, n, 0, sms), kMoveThreads, stream, set, src, dst, n, num_pages);
}

int gqa_pages_reserve(int32_t* block_table, const int32_t* seq_lens, int32_t* ref_counts, int32_t* counts,
                      int B, int max_pages_per_seq, int page_size, int num_pages, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
    int st = check_sizes(B, max_pages_per_seq, page_size, num_pages);
    if (st != GQA_OK) return st;
    if (B > GQA_MAX_PAGE_ROWS || (long long)B * max_pages_per_seq >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
    if (!block_table || !seq_lens || !ref_counts || !counts) return GQA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(ref_counts) || !aligned4(counts))
        return GQA_ERR_MISALIGNED;
    st = check_ws(workspace, workspace_bytes, B, num_pages);
    if (st != GQA_OK) return st;
    const size_t rows = 4 * (size_t)B, entries = rows * max_pages_per_seq, pages = 4 * (size_t)num_pages;
    const Range all[] = {{block_table, entries}, {seq_lens, rows}, {ref_counts, pages}, {counts, 8},
                         {workspace, gqa_pages_workspace_bytes(B, num_pages)}};
    if (overlap(all)) return GQA_ERR_INVALID_ARG;
    PagesParams p = {};
    p.lens = seq_lens;
    p.table_out = block_table;
    p.refs_out = ref_counts;
    p.counts = counts;
    p.ws = workspace;
    p.B = B;
    p.max_pages = max_pages_per_seq;
    p.page_size = page_size;
    p.num_pages = num_pages;
    return launch(reserve_kernel, kPlanCtas, kPlanThreads, stream, p);
}

int gqa_pages_fork(const gqa_page_pool_t* pools, int num_pools, const int32_t* src, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* ref_counts, int32_t* table_out, int32_t* lens_out,
                   int32_t* refs_out, int32_t* counts, int B, int max_pages_per_seq, int page_size,
                   int num_pages, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_sizes(B, max_pages_per_seq, page_size, num_pages);
    if (st != GQA_OK) return st;
    if (B > GQA_MAX_PAGE_ROWS) return GQA_ERR_UNSUPPORTED;
    PoolSet set;
    st = check_pools(pools, num_pools, num_pages, &set);
    if (st != GQA_OK) return st;
    if (!src || !block_table || !seq_lens || !ref_counts || !table_out || !lens_out || !refs_out || !counts)
        return GQA_ERR_INVALID_ARG;
    if (table_out == block_table || lens_out == seq_lens || refs_out == ref_counts) return GQA_ERR_INVALID_ARG;
    const size_t rows = 4 * (size_t)B, entries = rows * max_pages_per_seq, pages = 4 * (size_t)num_pages;
    const Range all[] = {{block_table, entries}, {seq_lens, rows}, {ref_counts, pages}, {src, rows},
                         {table_out, entries}, {lens_out, rows}, {refs_out, pages}, {counts, 8},
                         {workspace, gqa_pages_workspace_bytes(B, num_pages)}};
    if (!aligned4(src) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(ref_counts) ||
        !aligned4(table_out) || !aligned4(lens_out) || !aligned4(refs_out) || !aligned4(counts))
        return GQA_ERR_MISALIGNED;
    st = check_ws(workspace, workspace_bytes, B, num_pages);
    if (st != GQA_OK) return st;
    if (overlap(all)) return GQA_ERR_INVALID_ARG;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    const PagesParams p = {src, block_table, seq_lens, ref_counts, table_out, lens_out, refs_out, counts,
                           workspace, B, max_pages_per_seq, page_size, num_pages};
    st = launch(fork_plan_kernel, kPlanCtas, kPlanThreads, stream, p);
    if (st != GQA_OK) return st;
    return launch(fork_kernel, move_grid(set, B, (long long)B * max_pages_per_seq, sms), kMoveThreads, stream,
                  set, p);
}

int gqa_pages_free(const uint8_t* done, int32_t* block_table, int32_t* seq_lens, int32_t* ref_counts, int B,
                   int max_pages_per_seq, int num_pages, cudaStream_t stream) {
    const int st = check_sizes(B, max_pages_per_seq, 1, num_pages);
    if (st != GQA_OK) return st;
    if (!done || !block_table || !seq_lens || !ref_counts) return GQA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(ref_counts)) return GQA_ERR_MISALIGNED;
    const Range all[] = {{done, (size_t)B}, {block_table, 4 * (size_t)B * max_pages_per_seq}, {seq_lens, 4 * (size_t)B},
                         {ref_counts, 4 * (size_t)num_pages}};
    if (overlap(all)) return GQA_ERR_INVALID_ARG;
    int sms;
    unsigned* status;
    const int dv = current_device(&sms, &status);
    if (dv != GQA_OK) return dv;
    PagesParams p = {};
    p.table_out = block_table;
    p.lens_out = seq_lens;
    p.refs_out = ref_counts;
    p.B = B;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    PoolSet none;
    none.n = 0;
    return launch(free_kernel, move_grid(none, 0, (long long)B * max_pages_per_seq, sms), kMoveThreads, stream,
                  done, p);
}

int gqa_pages_compact(const gqa_page_pool_t* pools, int num_pools, const int32_t* block_table,
                      const int32_t* ref_counts, int32_t* table_out, int32_t* refs_out, int32_t* counts, int B,
                      int max_pages_per_seq, int num_pages, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
    int st = check_sizes(B, max_pages_per_seq, 1, num_pages);
    if (st != GQA_OK) return st;
    PoolSet set;
    st = check_pools(pools, num_pools, num_pages, &set);
    if (st != GQA_OK) return st;
    if (!block_table || !ref_counts || !table_out || !refs_out || !counts) return GQA_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(ref_counts) || !aligned4(table_out) || !aligned4(refs_out) ||
        !aligned4(counts))
        return GQA_ERR_MISALIGNED;
    st = check_ws(workspace, workspace_bytes, B, num_pages);
    if (st != GQA_OK) return st;
    // In place is the same array; of two ranges that are one, the second is left out.
    const size_t entries = 4 * (size_t)B * max_pages_per_seq, pages = 4 * (size_t)num_pages;
    const Range all[] = {{block_table, entries}, {ref_counts, pages}, {table_out, table_out == block_table ? 0 : entries},
                         {refs_out, refs_out == ref_counts ? 0 : pages}, {counts, 8},
                         {workspace, gqa_pages_workspace_bytes(B, num_pages)}};
    if (overlap(all)) return GQA_ERR_INVALID_ARG;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    PagesParams p = {};
    p.table = block_table;
    p.refs = ref_counts;
    p.table_out = table_out;
    p.refs_out = refs_out;
    p.counts = counts;
    p.ws = workspace;
    p.B = B;
    p.max_pages = max_pages_per_seq;
    p.num_pages = num_pages;
    st = launch(compact_plan_kernel, kPlanCtas, kPlanThreads, stream, p);
    if (st != GQA_OK) return st;
    return launch(compact_kernel, move_grid(set, num_pages / 2, (long long)B * max_pages_per_seq, sms),
                  kMoveThreads, stream, set, p);
}

}  // extern "C"
