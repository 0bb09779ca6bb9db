// How the attention of a packed batch is shared out over the CTAs. Plain
// arithmetic, the same on the device and on the host.
//
// A unit is (sequence, KV head, pair of 128-row tiles): 2 * tq new tokens, each
// with the H / G rows of its heads. Its length is the keys that its last token
// sees, plus a pad for what its start and end cost. All units lie end to end,
// sequence by sequence, KV head by KV head, and every CTA takes an equal share of
// that line. Where a boundary between shares falls inside a unit, its key tiles
// are cut there; the parts are merged afterwards.
#pragma once

#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace gqa {

constexpr int kRgTileShift = 7;
constexpr int kRgTile = 1 << kRgTileShift;   // rows of a tile, and keys of a key tile
// The times of this file are of one batch in a captured graph, in three orders of its
// sequences, one after another; calls from Python whose inputs change take up to 10 %
// longer.
//
// Least key tiles of a part of a unit: 8 prompts of 1024 (16 heads, D 64) take 43.9 us
// with two, 41.5 with four, 41.3 with six; 24 ragged ones (16 heads of their own, D 64)
// 161, 161 and 164; with 32/8 heads and D 128, and one of 16384, no difference.
constexpr int kRgMinPart = 4;
constexpr int kRgMinShare = 512;      // least share of a CTA, in keys: twice that was no faster

struct RgSeq {
    int start, n, T;                  // first row, new tokens, keys
};

struct RgUnit {
    int seq, g;
    int row0;                         // first token's row
    int tokens[2];                    // of tiles A and B
    int pos0;                         // position of the first token (below 0: sees nothing)
    int pos_last;                     // and of the last
    int key0;                         // packed: row of the sequence's first token
    int j0;                           // first key tile of this part
    int tiles[2];                     // key tiles of this part that A and B see
    int slot;                         // workspace slot of this part, -1: the unit is whole
    int first, parts;                 // CTAs [first, first + parts) hold the unit's parts
    int counter;                      // of the unit's arrivals
    int valid;                        // 0: no more units
};
static_assert(sizeof(RgUnit) == 64, "a unit is read as 16-byte words");

// Sizes that the line depends on: tokens of a tile, KV heads, and two weights.
// eighths: what a key of a unit with rows in tile A alone counts; its tiles go through
// both pipelines in turn. (A single token's tiles wait for copies, a short chunk's for
// products; one number serves both.) Chunks among single tokens (48 sequences, 32/8
// heads), D 128: 276 us with 6, 259 with 5, 286 with 4; D 64: 238, 223, 212 and 249 with
// 3 (16 heads of their own 273, 244, 224 and 241).
// pad: what a unit counts beyond its keys, for its start and end. 24 ragged prompts, D 128:
// 351 us with 256, 336 with 384, 348 with 512; D 64: 286 with 256, 293 with 320, 298 with
// 384 (16 heads of their own 161, 164, 169).
struct RgLine {
    int tq, G, eighths, pad;

    __host__ __device__ static RgLine of(int tq, int G, int D) {
        return D == 128 ? RgLine{tq, G, 5, 384} : RgLine{tq, G, 4, 256};
    }

    __host__ __device__ int pairs(int n) const { return (int)(((unsigned)n + 2u * tq - 1) / (2u * tq)); }
    __host__ __device__ static long long base(const RgSeq& s) { return s.T > s.n ? s.T - s.n : 0; }
    // Where pair pr of a KV head starts, from the head's start.
    __host__ __device__ long long start(const RgSeq& s, int pr) const {
        return pr * (base(s) + pad) + (long long)tq * pr * (pr + 1ll);
    }
    __host__ __device__ bool single(const RgSeq& s, int pr) const { return s.n - pr * 2 * tq <= tq; }
    __host__ __device__ long long length(const RgSeq& s, int pr) const {
        const long long seen = (pr + 1ll) * 2 * tq, keys = base(s) + (seen < s.n ? seen : s.n);
        return (single(s, pr) ? keys * eighths >> 3 : keys) + pad;
    }
    // Keys of such a unit by their length on the line (8 / 5 as 410 / 256).
    __host__ __device__ long long keys_of(long long y) const { return eighths == 5 ? y * 410 >> 8 : 2 * y; }
    // Of one KV head.
    __host__ __device__ long long head(const RgSeq& s) const {
        const int P = pairs(s.n);
        return P == 0 ? 0 : start(s, P - 1) + length(s, P - 1);
    }
    __host__ __device__ int pair_at(const RgSeq& s, long long y) const {
        int lo = 0, hi = pairs(s.n) - 1;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (start(s, mid) <= y) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
};

// The shares: CTA c takes [at(c), at(c + 1)) of the line.
struct RgShares {
    long long each, more;             // `more` CTAs take one key more
    int ctas;

    __host__ __device__ static RgShares of(long long total, int grid) {
        long long c = total / kRgMinShare;
        if (c > grid) c = grid;
        if (c < 1) c = 1;
        // (64-bit division takes long)
        const long long each = total >> 31 == 0 ? (long long)((unsigned)total / (unsigned)c) : total / c;
        return {each, total - each * c, (int)c};
    }
    __host__ __device__ long long at(int c) const { return each * c + (c < more ? c : more); }
};

// Fills the part of unit (s, g, pr), which starts at `at` on the line, that CTA c
// takes; false if it takes none.
__host__ __device__ __forceinline__ bool rg_unit(const RgLine& line, const RgShares& sh, int c, const RgSeq& s, int pr,
                                                 long long at, RgUnit* u) {
    const int q2 = 2 * line.tq;
    const int left = s.n - pr * q2;
    const int a = left < line.tq ? left : line.tq;
    const int b = left < q2 ? left - a : line.tq;
    const int pos0 = s.T - s.n + pr * q2;
    const int lim_a = pos0 + a - 1, lim_b = pos0 + a + b - 1;
    const int tiles_a = lim_a < 0 ? 0 : (lim_a >> kRgTileShift) + 1;
    const int tiles_b = b == 0 || lim_b < 0 ? 0 : (lim_b >> kRgTileShift) + 1;
    const int tiles = tiles_b > tiles_a ? tiles_b : tiles_a;
    const long long len = line.length(s, pr);
    const bool alone = line.single(s, pr);
    // Key tile that a boundary x cuts at. Parts below kRgMinPart tiles go to the neighbour.
    auto cut = [&](long long x) {
        const long long y = x - at;
        if (y <= 0) return 0;
        if (y >= len) return tiles;
        const long long t = ((alone ? line.keys_of(y) : y) + kRgTile / 2) >> kRgTileShift;
        if (t < kRgMinPart) return 0;
        return t > tiles - kRgMinPart ? tiles : (int)t;
    };
    // The CTAs with parts of the unit are neighbours: where they begin and end.
    int first = c, last = c, j0 = 0, j1 = 0;
    for (int t; (t = cut(sh.at(first))) > 0; --first)
        if (first == c) j0 = t;
    for (;; ++last) {
        const int t = cut(sh.at(last + 1));
        if (last == c) j1 = t;
        if (t == tiles) break;
    }
    if (tiles == 0 ? at < sh.at(c) || at >= sh.at(c + 1) : j0 >= j1) return false;
    u->row0 = s.start + pr * q2;
    u->tokens[0] = a;
    u->tokens[1] = b;
    u->pos0 = pos0;
    u->pos_last = lim_b;
    u->key0 = s.start;
    u->j0 = j0;
    const int ea = tiles_a < j1 ? tiles_a : j1, eb = tiles_b < j1 ? tiles_b : j1;
    u->tiles[0] = ea > j0 ? ea - j0 : 0;
    u->tiles[1] = eb > j0 ? eb - j0 : 0;
    u->valid = 1;
    const bool whole = tiles == 0 || first == last;
    u->slot = whole ? -1 : 2 * c + (at < sh.at(c) ? 0 : 1);
    u->first = whole ? c : first;
    u->parts = whole ? 1 : last - first + 1;
    u->counter = whole ? 0 : 2 * first + (at < sh.at(first) ? 0 : 1);
    return true;
}

}  // namespace gqa
