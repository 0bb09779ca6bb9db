// Parameters and launch interface of the paged e4m3 attention kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace gqa {

constexpr int kP8Tokens = 128;     // tokens per tile: one per thread of a softmax group, M of the products
// Fewest tiles of a split unit worth a CTA: a tile takes 0.5 us, handing a part
// over and merging it 3.2 us.
constexpr int kP8MinTiles = 8;
constexpr int kP8MaxRows = 32;     // query rows of a unit; more are further units

// Division of n < 2^31 by a fixed d >= 1: (n * mul / 2^32 + n) / 2^shift.
struct FastDiv {
    unsigned mul;
    int shift;
    explicit FastDiv(unsigned d = 1) : mul(0), shift(0) {
        while ((1u << shift) < d) ++shift;
        mul = (unsigned)((((1ull << shift) - d) << 32) / d + 1);
    }
    __host__ __device__ int operator()(int n) const {
        const unsigned high = (unsigned)(((unsigned long long)(unsigned)n * mul) >> 32);
        return (int)((high + (unsigned)n) >> shift);
    }
};

struct PagedFp8Params {
    const uint16_t* q;         // [B, sq, H, D] bf16
    const float* k_scale;      // [num_pages, G, blocks]
    const float* v_scale;
    const int32_t* table;      // [B, max_pages]
    const int32_t* lens;       // [B]
    uint16_t* out;             // [B, sq, H, D] bf16
    float* lse;                // [B, sq, H] or nullptr
    unsigned long long* counters;   // [grid][2]: arrivals of the unit that a CTA's share starts
    unsigned long long tag;    // of this call, in the counters (48 bits)
    float* part;               // [grid][2][slot]: O[rows][D], m[rows], l[rows]
    unsigned* status;
    unsigned long long wait_timeout_ns;
    float scale_log2;
    int B, sq, H, G, R, heads_per_group, row_tiles;
    FastDiv by_heads, by_row_tiles;   // by heads_per_group and row_tiles
    int page_shift, num_pages, max_pages, blocks;
    int small_plan;            // up to 128 entries (b, row tile), 32-bit tile arithmetic
    int skip_tile;             // fault injection for tests (-1: off)
};

struct PagedFp8Launch {
    CUtensorMap tm_k, tm_v;    // [num_pages * G][page_size][D] bytes
    PagedFp8Params p;
    int grid;
    cudaStream_t stream;
};

inline int p8_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : kP8MaxRows; }
// Tiles that a unit counts beyond its own where the units are not alike: what its
// end (its output, the next one's queries) costs the CTA. GB/s with 512 units of
// 512 to 32768 | of up to 4096 tokens, pad by pad: 32 rows 0: 5820 | 1830, 4: 6260 |
// 2460, 8: 6460 | 2980, 12: 6400 | 3060; 16 rows 4: 6930 | 3260, 6: 6900 | 3550, 8: 6860 |
// 3760; 8 rows 0: 6920 | 3210, 4: 7010 | 5150, 8: 6960 | 5130 (300 sequences 0:
// 6330, 4: 6680, 8: 6460).
__host__ __device__ constexpr int p8_unit_pad(int rows) { return rows == 32 ? 8 : rows == 16 ? 6 : 4; }

// CTAs of a call: one per SM, fewer if even full tables hold less work.
inline long long p8_table_tiles(int page_size, int max_pages) {
    return ((long long)max_pages * page_size + kP8Tokens - 1) / kP8Tokens;
}
inline int p8_grid(int B, int G, int R, int page_size, int max_pages, int sms) {
    const int rows = p8_rows(R);
    const long long units = (long long)B * G * ((R + rows - 1) / rows);
    const long long split = units * p8_table_tiles(page_size, max_pages) / kP8MinTiles;
    const long long want = split > units ? split : units;
    return (int)(want < sms ? want : sms);
}
// Whether every warp plans by itself: up to 128 entries (b, row tile), and
// products of tiles and CTAs that fit 32 bits.
inline bool p8_small(int B, int G, int R, int page_size, int max_pages, int grid) {
    const int rows = p8_rows(R);
    const long long entries = (long long)B * ((R + rows - 1) / rows);
    return entries <= 128 && entries * G * (p8_table_tiles(page_size, max_pages) + p8_unit_pad(rows)) <
                                 (1ll << 32) / (grid + 1);
}

__host__ __device__ inline size_t p8_slot_floats(int rows, int D) { return (size_t)rows * D + 2 * rows; }

cudaError_t launch_paged_fp8_d64(const PagedFp8Launch& a);
cudaError_t launch_paged_fp8_d128(const PagedFp8Launch& a);

}  // namespace gqa
