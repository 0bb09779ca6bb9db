// C ABI of gqa_decode_paged_fp8: argument checks, the grid, TMA descriptors and
// the launch. The kernels are in gqa_paged_fp8.cuh.
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_decode.h"
#include "gqa_launch.h"
#include "gqa_paged_fp8.h"

using namespace gqa;

namespace {

int check_paged_fp8(int B, int sq, int H, int G, int D, int page_size, int max_pages) {
    if (B <= 0 || sq <= 0 || H <= 0 || G <= 0 || D <= 0 || page_size <= 0 || max_pages <= 0)
        return GQA_ERR_INVALID_ARG;
    if (H % G != 0) return GQA_ERR_HEAD_RATIO;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1))) return GQA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size >= (1ll << 31) - 128 || (long long)B * sq * H >= (1ll << 31))
        return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

size_t counter_bytes(int grid) { return (sizeof(unsigned long long) * 2 * (size_t)grid + 255) & ~size_t(255); }

size_t paged_fp8_ws_bytes(int grid, int R, int D) {
    return counter_bytes(grid) + sizeof(float) * 2 * (size_t)grid * p8_slot_floats(p8_rows(R), D);
}

}  // namespace

extern "C" {

size_t gqa_decode_paged_fp8_workspace_bytes(int B, int sq, int H, int G, int D, int page_size,
                                            int max_pages_per_seq) {
    if (check_paged_fp8(B, sq, H, G, D, page_size, max_pages_per_seq) != GQA_OK) return 0;
    int sms;
    unsigned* status;
    if (current_device(&sms, &status) != GQA_OK) return 0;
    const int R = H / G * sq;
    return paged_fp8_ws_bytes(p8_grid(B, G, R, page_size, max_pages_per_seq, sms), R, D);
}

int gqa_decode_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                         const float* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                         float scale, void* out, float* lse, int B, int sq, int H, int G, int D,
                         int page_size, int num_pages, int max_pages_per_seq, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
    int st = check_paged_fp8(B, sq, H, G, D, page_size, max_pages_per_seq);
    if (st != GQA_OK) return st;
    if (num_pages <= 0 || !(scale == scale) || scale - scale != 0.f) return GQA_ERR_INVALID_ARG;
    if ((long long)num_pages * G >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seq_lens || !out)
        return GQA_ERR_INVALID_ARG;
    const uintptr_t wide = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pages) |
                           reinterpret_cast<uintptr_t>(v_pages) | reinterpret_cast<uintptr_t>(out);
    const uintptr_t word = reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
                           reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
                           reinterpret_cast<uintptr_t>(lse);
    if ((wide & 15u) || (word & 3u)) return GQA_ERR_MISALIGNED;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    const int R = H / G * sq;
    const int grid = p8_grid(B, G, R, page_size, max_pages_per_seq, sms);
    if (!workspace || workspace_bytes < paged_fp8_ws_bytes(grid, R, D) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return GQA_ERR_WORKSPACE;
    PagedFp8Launch a;
    const int box = page_size < kP8Tokens ? page_size : kP8Tokens;
    st = encode_byte_map(&a.tm_k, k_pages, (long long)num_pages * G, page_size, D, box);
    if (st != GQA_OK) return st;
    st = encode_byte_map(&a.tm_v, v_pages, (long long)num_pages * G, page_size, D, box);
    if (st != GQA_OK) return st;
    PagedFp8Params& p = a.p;
    p.q = static_cast<const uint16_t*>(q);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = block_table;
    p.lens = seq_lens;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.counters = static_cast<unsigned long long*>(workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + counter_bytes(grid));
    p.tag = call_tag();
    p.status = status;
    wait_knobs(&p.wait_timeout_ns, &p.skip_tile);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.B = B;
    p.sq = sq;
    p.H = H;
    p.G = G;
    p.R = R;
    p.heads_per_group = H / G;
    p.row_tiles = (R + p8_rows(R) - 1) / p8_rows(R);
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    p.blocks = (page_size + 63) / 64;
    p.by_heads = FastDiv((unsigned)p.heads_per_group);
    p.by_row_tiles = FastDiv((unsigned)p.row_tiles);
    p.small_plan = p8_small(B, G, R, page_size, max_pages_per_seq, grid);
    a.grid = grid;
    a.stream = stream;
    const cudaError_t e = D == 64 ? launch_paged_fp8_d64(a) : launch_paged_fp8_d128(a);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

}  // extern "C"
