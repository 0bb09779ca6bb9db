// Parameters and launch interface of the paged e4m3 attention kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace gqa {

constexpr int kP8Tokens = 128;     // tokens per tile: one per thread of a softmax group, M of the products
constexpr int kP8MinTiles = 2;     // fewest tiles worth a CTA
constexpr int kP8MaxRows = 32;     // query rows of a unit; more are further units

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
    int page_shift, num_pages, max_pages, blocks;
    int small_plan;            // up to 128 entries (b, row tile), 32-bit tile arithmetic
    int even_ctas;             // grid for equal lengths (small plans)
    int skip_tile;             // fault injection for tests (-1: off)
};

struct PagedFp8Launch {
    CUtensorMap tm_k, tm_v;    // [num_pages * G][page_size][D] bytes
    PagedFp8Params p;
    int grid;
    cudaStream_t stream;
};

inline int p8_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : kP8MaxRows; }
__host__ __device__ inline size_t p8_slot_floats(int rows, int D) { return (size_t)rows * D + 2 * rows; }

cudaError_t launch_paged_fp8_d64(const PagedFp8Launch& a);
cudaError_t launch_paged_fp8_d128(const PagedFp8Launch& a);

}  // namespace gqa
