// Who computes what in the paged e4m3 attention: the tiles of all units, end to
// end, in equal shares, one per CTA. No instruction here is special to the
// kernel, so that the plan compiles for the host as well (with the warp's
// intrinsics given), where every share can be checked against every other.
#pragma once

#include "gqa_paged_fp8.h"

namespace gqa {

constexpr int kP8LenCopy = 384;           // sequences whose lengths a CTA keeps

// Lengths, from the CTA's copy where the batch fits it, and the tiles that the
// rows of an entry (b, row tile) see: with one row tile, all of the sequence's.
template <int RP>
struct P8Lens {
    const PagedFp8Params& p;
    int* copy;
    __device__ int global(int b) const {
        const int t = p.lens[b], most = p.max_pages << p.page_shift;
        return t < 0 ? 0 : (t > most ? most : t);
    }
    // One copy for all warps: of all sequences, or of those from the first one of
    // the CTA's share on. With 32 rows (and no register to spare) only the former:
    // the latter took lengths up to 4096 from 76 to 83 us; with 8 rows 1500
    // sequences gained, 777 to 659 us.
    __device__ int tokens(int b) const {
        if constexpr (RP == 32) return p.B <= kP8LenCopy ? copy[b] : global(b);
        const unsigned i = (unsigned)(b - copy[kP8LenCopy + 1]);
        return i < kP8LenCopy ? copy[i] : global(b);
    }
    __device__ void split(int entry, int& b, int& rt) const {
        b = p.by_row_tiles(entry);
        rt = entry - b * p.row_tiles;
    }
    __device__ int tiles(int entry) const {
        int b, rt;
        split(entry, b, rt);
        const int T = tokens(b);
        if (p.row_tiles == 1) return (T + kP8Tokens - 1) / kP8Tokens;
        const int last = min(p.R, (rt + 1) * RP) - 1;
        const int lim = T - p.sq + p.by_heads(last);
        return lim < 0 ? 0 : lim / kP8Tokens + 1;
    }
    // Tiles that a unit counts beyond its own in the plan.
    __device__ int pad() const { return copy[kP8LenCopy]; }
};

// A CTA's share as a run of segments of units.
struct P8Segment {
    int entry, g, i0, i1, n;     // tiles [i0, i1) of the unit's n
};
template <int RP>
struct P8Walk {
    long long left;              // of the CTA's share, padding included
    int entry, g, off;
    __device__ bool next(const P8Lens<RP>& lens, P8Segment& s) {
        if (left <= 0) return false;
        int n;
        if constexpr (RP == 32) {
            n = lens.tiles(entry);
            while (n == 0) {
                if (++entry >= lens.p.B * lens.p.row_tiles) return false;   // not while the lengths stay
                n = lens.tiles(entry);
            }
        } else {                      // the same; 8 rows, lengths up to 4096: 55 -> 51 us
            n = 0;
            while (n == 0) {
                if (entry >= lens.p.B * lens.p.row_tiles) return false;
                n = lens.tiles(entry);
                if (n == 0) ++entry;
            }
        }
        s.entry = entry;
        s.g = g;
        s.i0 = off;
        s.i1 = left < n - off ? off + (int)left : n;
        s.n = n;
        left -= s.i1 - s.i0 + lens.pad();
        off = 0;
        if (++g == lens.p.G) {
            g = 0;
            ++entry;
        }
        return true;
    }
};

struct P8Plan {
    long long total, begin, end;   // tiles of the call, and this CTA's, padding included
    long long left;                // of the latter from the first tile on
    int entry, g, off;             // where it begins
    int ctas;                      // CTAs that share the tiles
    // What is left of the share: nothing of an empty one, wherever it would begin;
    // one that begins in a unit's padding begins with the next unit.
    __device__ void skip_pad(int n, int pad, int G) {
        left = end - begin;
        if (left <= 0 || off < n) return;
        left -= n + pad - off;
        off = 0;
        if (++g == G) {
            g = 0;
            ++entry;
        }
    }
    // The CTA whose share holds tile t of the call; in 32 bits where both sides fit.
    __device__ int owner(long long t) const {
        const unsigned long long x = (unsigned long long)(t + 1) * (unsigned)ctas - 1;
        const unsigned long long of = (unsigned long long)total;
        return (x | of) >> 32 ? (int)(x / of) : (int)((unsigned)x / (unsigned)of);
    }
    // The CTAs c0 .. c0 + n - 1 share the unit of a segment of this CTA's that is
    // not the whole of it: one that began in another CTA, or goes on in one.
    __device__ __forceinline__ void sharers(const P8Segment& s, int& c0, int& n) const {
        const long long unit0 = s.i0 > 0 ? begin - s.i0 : end - s.i1;
        c0 = owner(unit0);
        n = owner(unit0 + s.n - 1) - c0 + 1;
    }
};

// Up to 128 entries, and 32-bit products of tiles and CTAs: every warp finds
// the CTA's share by itself, four entries a lane, from the CTA's one copy of
// the lengths (all warps have to walk the same tiles).
template <int RP>
__device__ __forceinline__ P8Plan p8_small_plan(const P8Lens<RP>& lens) {
    const PagedFp8Params& p = lens.p;
    const int lane = threadIdx.x & 31;
    const int entries = p.B * p.row_tiles;
    unsigned n[4], mine = 0;
    if (p.row_tiles == 1) {
        const int4 T = reinterpret_cast<const int4*>(lens.copy)[lane];      // 0 past the batch
        n[0] = ((unsigned)T.x + kP8Tokens - 1) / kP8Tokens;
        n[1] = ((unsigned)T.y + kP8Tokens - 1) / kP8Tokens;
        n[2] = ((unsigned)T.z + kP8Tokens - 1) / kP8Tokens;
        n[3] = ((unsigned)T.w + kP8Tokens - 1) / kP8Tokens;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = lane * 4 + k < entries ? (unsigned)lens.tiles(lane * 4 + k) : 0;
    }
    unsigned lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mine += n[k];
        if (lane * 4 + k < entries) lo = min(lo, n[k]), hi = max(hi, n[k]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    const bool equal = lo == hi;                  // the same in every lane, as all that follows
    // A CTA for every unit, or for every eight tiles.
    const unsigned tiles = __reduce_add_sync(0xffffffffu, mine) * (unsigned)p.G;
    const unsigned units = (unsigned)entries * p.G;
    unsigned ctas = min(min(gridDim.x, max(units, tiles / kP8MinTiles)), max(tiles, 1u));
    // Equal lengths: whole units per CTA, or the same number of CTAs per unit,
    // where that keeps four fifths of them; no unit is then cut unevenly.
    if (equal && hi > 0) {
        const unsigned per = (units + ctas - 1) / ctas;
        const unsigned even = per > 1 ? (units % per == 0 ? units / per : 0) : units * (ctas / units);
        if (5 * even >= 4 * ctas) ctas = even;
    }
    // Otherwise a unit counts some tiles more, for what its end costs a CTA.
    const unsigned pad = equal ? 0 : p8_unit_pad(RP);
    unsigned total, before;
    if (equal) {
        total = tiles;
        before = (unsigned)min(lane * 4, entries) * hi * (unsigned)p.G;
    } else {
        mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (n[k]) n[k] += pad;
            mine += n[k];
        }
        unsigned x = mine * (unsigned)p.G;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        total = __shfl_sync(0xffffffffu, x, 31);
        before = x - mine * (unsigned)p.G;
    }
    mine *= (unsigned)p.G;
    const unsigned c = blockIdx.x;
    const unsigned t0 = c < ctas ? total * c / ctas : total, t1 = c < ctas ? total * (c + 1) / ctas : total;
    // The lane whose entries hold tile t0, and where in them it lies.
    const unsigned here = __ballot_sync(0xffffffffu, t0 >= before && t0 < before + mine);
    int e = lane * 4;
    unsigned at = before, ne = n[0];
#pragma unroll
    for (int k = 1; k < 4; ++k)
        if (at + ne * p.G <= t0) {
            at += ne * p.G;
            ne = n[k];
            ++e;
        }
    const unsigned in = t0 - at, g = ne ? in / ne : 0;
    const int src = here ? __ffs(here) - 1 : 0;
    P8Plan plan;
    plan.total = total;
    plan.begin = t0;
    plan.end = t1;
    plan.entry = __shfl_sync(0xffffffffu, e, src);
    plan.g = __shfl_sync(0xffffffffu, (int)g, src);
    plan.off = __shfl_sync(0xffffffffu, (int)(in - g * ne), src);
    plan.ctas = (int)ctas;
    plan.skip_pad(__shfl_sync(0xffffffffu, (int)(ne - pad), src), (int)pad, p.G);
    if (lane == 0) lens.copy[kP8LenCopy] = (int)pad;        // copy[kP8LenCopy + 1] is the caller's
    __syncwarp();
    return plan;
}

// a * b / c for 64-bit a, in 32 bits where they do.
__device__ __forceinline__ long long muldiv(long long a, int b, int c) {
    const unsigned long long x = (unsigned long long)a * (unsigned)b;
    return x >> 32 ? (long long)(x / (unsigned)c) : (long long)((unsigned)x / (unsigned)c);
}

// Any sizes, all threads: sums the tiles of all entries, each thread over a
// contiguous range of them, and finds where this CTA's share begins. The
// caller synchronises the CTA before anyone reads the plan.
template <int RP, int THREADS>
__device__ __noinline__ void p8_make_plan(const PagedFp8Params& p, int* len_copy, P8Plan* plan, long long* warp_sum) {
    const P8Lens<RP> lens = {p, len_copy};
    const int entries = p.B * p.row_tiles;
    const int per = (entries + THREADS - 1) / THREADS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.B <= kP8LenCopy)
        for (int b = threadIdx.x; b < p.B; b += THREADS) len_copy[b] = lens.global(b);
    if (threadIdx.x == 0) {
        len_copy[kP8LenCopy] = p8_unit_pad(RP);
        len_copy[kP8LenCopy + 1] = p.B <= kP8LenCopy ? 0 : p.B;   // none yet
        *plan = P8Plan{};
    }
    __syncthreads();
    const int e0 = (int)min((long long)entries, (long long)threadIdx.x * per), e1 = min(entries, e0 + per);
    long long mine = 0;
    auto padded = [&](int e) {
        const int n = lens.tiles(e);
        return n ? n + p8_unit_pad(RP) : 0;
    };
    for (int e = e0; e < e1; ++e) mine += padded(e);
    mine *= p.G;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    const long long most = max((long long)entries * p.G, total / kP8MinTiles);
    const int ctas = (int)max(1ll, min(min((long long)gridDim.x, most), total));
    const int c = blockIdx.x;
    const long long t0 = c < ctas ? muldiv(total, c, ctas) : total;
    const long long t1 = c < ctas ? muldiv(total, c + 1, ctas) : total;
    if (t0 < t1 ? t0 >= before && t0 < before + mine : threadIdx.x == 0) {
        plan->total = total;
        plan->begin = t0;
        plan->end = t1;
        plan->ctas = ctas;
        plan->entry = plan->g = plan->off = 0;
        plan->left = 0;
        if (t0 < t1) {
            long long at = before;
            int e = e0, n = padded(e);
            while (at + (long long)n * p.G <= t0) {
                at += (long long)n * p.G;
                n = padded(++e);
            }
            plan->entry = e;
            plan->g = (int)((t0 - at) / n);
            plan->off = (int)((t0 - at) % n);
            plan->skip_pad(n - p8_unit_pad(RP), p8_unit_pad(RP), p.G);
        }
    }
    if (RP < 32 && p.B > kP8LenCopy) {
        __syncthreads();
        const int first = p.by_row_tiles(plan->entry);
        for (int i = threadIdx.x; i < kP8LenCopy && first + i < p.B; i += THREADS) len_copy[i] = lens.global(first + i);
        if (threadIdx.x == 0) len_copy[kP8LenCopy + 1] = first;
    }
}

}  // namespace gqa
