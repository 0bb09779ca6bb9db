// Parameters and launch interface of the attention of packed batches.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "gqa_paged_fp8.h"

namespace gqa {

constexpr int kRgUnits = 4;              // units that a CTA has under way at most

struct RaggedParams {
    const int32_t* cu;         // [B + 1]
    const int32_t* lens;       // [B], paged only
    const int32_t* table;      // [B, max_pages], paged only
    uint16_t* out;             // [N, H, D] bf16
    float* lse;                // [N, H] or nullptr
    unsigned long long* counters;   // [grid][2]: arrivals of split units
    int* bad;                  // [grid][kRgUnits][D]: first positions of values that are not finite
    float* part;               // [grid][2][slot]: O[256][D], m[256], l[256]
    unsigned long long tag;    // of this call, in the counters (48 bits)
    unsigned* status;
    unsigned long long wait_timeout_ns;
    float scale_log2;
    int N, B, H, G, heads_per_group, tq;   // tq: tokens of a 128-row tile
    FastDiv by_heads;          // by heads_per_group
    int page_shift, num_pages, max_pages;
    int wide;                  // out is 32-byte aligned
    int skip_tile;             // fault injection for tests (-1: off)
};

struct RaggedLaunch {
    // q [N][H][D]; k, v [N][G][D] or, paged, [num_pages * G][page_size][D]
    CUtensorMap tm_q, tm_k, tm_v;
    RaggedParams p;
    int grid;
    cudaStream_t stream;
};

inline size_t rg_bad_bytes(int D, int grid) { return sizeof(int) * kRgUnits * (size_t)D * grid; }
// A part's O, m and l: 256 rows of both tiles.
__host__ __device__ constexpr size_t rg_slot_floats(int D) { return (size_t)256 * (D + 2); }
inline size_t rg_counter_bytes(int grid) { return (sizeof(unsigned long long) * 2 * (size_t)grid + 255) & ~size_t(255); }

cudaError_t launch_ragged_d64(const RaggedLaunch& a, bool paged);
cudaError_t launch_ragged_d128(const RaggedLaunch& a, bool paged);

}  // namespace gqa
