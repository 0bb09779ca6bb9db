// Internal interface between the C ABI (api.cu) and the kernel translation
// units (one per head dimension, so that they compile in parallel).
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>

#include "gqa_common.h"

namespace gqa {

struct LaunchArgs {
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    DecodeParams p;
    int row_tiles;   // 1 or 2
    bool kv8;        // fp8 e4m3 K/V codes with per-tile scales
    bool pdl;        // launch with programmatic stream serialization
    cudaStream_t stream;
};

// Enqueue the split-KV kernel (one launch per decode step) for D = 64 / D = 128.
cudaError_t launch_d64(const LaunchArgs& a);
cudaError_t launch_d128(const LaunchArgs& a);
cudaError_t launch_d128_fp8(const LaunchArgs& a);

// The prefill kernel: one CTA per 128-row tile of one (sequence, KV head).
struct PrefillLaunchArgs {
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    PrefillParams p;
    unsigned grid;
    cudaStream_t stream;
    bool pdl;        // the combine: launch with programmatic stream serialization
};
cudaError_t launch_prefill(int D, const PrefillLaunchArgs& a);   // + the combine when split
size_t prefill_workspace_bytes(int D, long long items, int splits);
int prefill_smem_bytes(int D);

// Dynamic shared memory and threads per CTA of the split-KV kernel.
int splitkv_smem_bytes(int D, int row_tiles, bool kv8 = false);
int splitkv_threads(int D, int row_tiles, bool kv8 = false);
int splitkv_stages(int D, int row_tiles, bool kv8 = false);

// Host services of api.cu for the entry points of the other translation units.
int remember_cuda_error(cudaError_t e);                     // returns GQA_ERR_CUDA
int current_device(int* sms, unsigned** status);            // SM count, status word
unsigned long long call_tag();                              // 48 bits, another for every call
void wait_knobs(unsigned long long* timeout_ns, int* skip_tile);
// cuTensorMapEncodeTiled of a 3-D uint8 tensor [slabs][rows][cols] (dense) with
// boxes of box_rows x cols bytes and the swizzle that `cols` (64 or 128) spans.
int encode_byte_map(CUtensorMap* map, const void* base, long long slabs, int rows, int cols, int box_rows);
// The same of a bf16 cache [slabs][rows][D] with boxes of box_rows x 64 elements.
int encode_page_map(CUtensorMap* map, const void* base, long long slabs, int rows, int D, int box_rows);
// And of packed bf16 rows [N][heads][D], tokens `stride` elements apart, with boxes
// of box_tokens x box_heads x 64 elements.
int encode_rows_map(CUtensorMap* map, const void* base, int N, int heads, int D, long long stride, int box_heads,
                    int box_tokens);

}  // namespace gqa
