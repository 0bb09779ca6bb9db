// C ABI of the attention of packed batches (gqa_prefill_packed, gqa_prefill_paged):
// argument checks, TMA descriptors and the launch. The kernels are in
// gqa_ragged.cuh.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gqa_decode.h"
#include "gqa_launch.h"
#include "gqa_ragged.h"
#include "gqa_ragged_plan.cuh"

namespace gqa {
namespace {

bool aligned(const void* x, unsigned mask) { return (reinterpret_cast<uintptr_t>(x) & mask) == 0; }

constexpr float kLog2E = 1.4426950408889634f;     // exponentials are of base 2
bool usable(float scale) { return scale > 0.f && std::isfinite(scale * kLog2E); }

int check_sizes(int N, int B, int H, int G, int D) {
    if (N < 0 || B <= 0 || H <= 0 || G <= 0 || D <= 0) return GQA_ERR_INVALID_ARG;
    if (H % G != 0) return GQA_ERR_HEAD_RATIO;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (H / G > 128 || (long long)N * H >= (1ll << 31) || B >= (1 << 24) || (long long)B * G >= (1 << 30)) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

int check_rows(const void* x, long long stride, int heads, int D) {
    if (stride < (long long)heads * D) return GQA_ERR_INVALID_ARG;
    if (!aligned(x, 15u) || (stride & 7)) return GQA_ERR_MISALIGNED;
    return stride >= (1ll << 38) ? GQA_ERR_UNSUPPORTED : GQA_OK;
}

// One CTA per SM; the device's plan gives work to as many as there is work for. The
// binding relies on it that N, B, H and G do not matter.
size_t workspace_need(int D, int grid) {
    return rg_counter_bytes(grid) + rg_bad_bytes(D, grid) + sizeof(float) * 2 * grid * rg_slot_floats(D);
}

struct Call {
    RaggedLaunch a = {};
};

// Fills what both calls share; q's descriptor, workspace and knobs.
int begin(Call& c, const void* q, const int32_t* cu, float scale, void* out, float* lse, int N, int B, int H, int G,
          int D, long long q_stride, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int sms;
    RaggedParams& p = c.a.p;
    int st = current_device(&sms, &p.status);
    if (st != GQA_OK) return st;
    c.a.grid = sms;
    if (!workspace || workspace_bytes < workspace_need(D, sms) || !aligned(workspace, 255u)) return GQA_ERR_WORKSPACE;
    const int r = H / G, tq = 128 / r;
    if ((st = encode_rows_map(&c.a.tm_q, q, N, H, D, q_stride, r, tq)) != GQA_OK) return st;
    p.cu = cu;
    p.out = static_cast<uint16_t*>(out);
    p.wide = aligned(out, 31u);
    p.lse = lse;
    p.counters = static_cast<unsigned long long*>(workspace);
    p.bad = reinterpret_cast<int*>(static_cast<char*>(workspace) + rg_counter_bytes(sms));
    p.part = reinterpret_cast<float*>(reinterpret_cast<char*>(p.bad) + rg_bad_bytes(D, sms));
    p.tag = call_tag();
    wait_knobs(&p.wait_timeout_ns, &p.skip_tile);
    p.scale_log2 = scale * kLog2E;
    p.N = N;
    p.B = B;
    p.H = H;
    p.G = G;
    p.heads_per_group = r;
    p.tq = tq;
    p.by_heads = FastDiv((unsigned)r);
    c.a.stream = stream;
    return GQA_OK;
}

int launch(const Call& c, int D, bool paged) {
    const cudaError_t e = D == 64 ? launch_ragged_d64(c.a, paged) : launch_ragged_d128(c.a, paged);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_prefill_ragged_workspace_bytes(int N, int B, int H, int G, int D) {
    if (check_sizes(N, B, H, G, D) != GQA_OK) return 0;
    int sms;
    unsigned* status;
    if (current_device(&sms, &status) != GQA_OK) return 0;
    return workspace_need(D, sms);
}

int gqa_prefill_packed(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, float scale,
                       void* out, float* lse, int N, int B, int H, int G, int D, long long q_stride,
                       long long k_stride, long long v_stride, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    int st = check_sizes(N, B, H, G, D);
    if (st != GQA_OK) return st;
    if (N == 0) return GQA_OK;              // tensors without rows have no address
    if (!q || !k || !v || !cu_seqlens || !out || !usable(scale)) return GQA_ERR_INVALID_ARG;
    if ((st = check_rows(q, q_stride, H, D)) != GQA_OK || (st = check_rows(k, k_stride, G, D)) != GQA_OK ||
        (st = check_rows(v, v_stride, G, D)) != GQA_OK)
        return st;
    if (!aligned(out, 15u) || !aligned(cu_seqlens, 3u) || !aligned(lse, 3u)) return GQA_ERR_MISALIGNED;
    Call c;
    st = begin(c, q, cu_seqlens, scale, out, lse, N, B, H, G, D, q_stride, workspace, workspace_bytes, stream);
    if (st != GQA_OK) return st;
    // No more CTAs than the rows have work for: all in one sequence, and the most that
    // cutting them into B leaves over.
    const RgLine line = RgLine::of(c.a.p.tq, G, D);
    const long long most = (line.head({0, N, N}) + (long long)B * (line.pad + 2 * c.a.p.tq)) * G / kRgMinShare + 1;
    if (most < c.a.grid) c.a.grid = (int)most;
    if ((st = encode_rows_map(&c.a.tm_k, k, N, G, D, k_stride, 1, 128)) != GQA_OK) return st;
    if ((st = encode_rows_map(&c.a.tm_v, v, N, G, D, v_stride, 1, 128)) != GQA_OK) return st;
    return launch(c, D, false);
}

int gqa_prefill_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                      const int32_t* cu_new, const int32_t* seq_lens, float scale, void* out, float* lse, int N,
                      int B, int H, int G, int D, long long q_stride, int page_size, int num_pages,
                      int max_pages_per_seq, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_sizes(N, B, H, G, D);
    if (st != GQA_OK) return st;
    if (N == 0) return GQA_OK;              // tensors without rows have no address
    if (!q || !k_pages || !v_pages || !block_table || !cu_new || !seq_lens || !out || !usable(scale) ||
        page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0)
        return GQA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1))) return GQA_ERR_UNSUPPORTED;
    if ((long long)max_pages_per_seq * page_size >= (1ll << 31) - 128 || (long long)num_pages * G >= (1ll << 31) - 1)
        return GQA_ERR_UNSUPPORTED;
    if ((st = check_rows(q, q_stride, H, D)) != GQA_OK) return st;
    if (!aligned(k_pages, 15u) || !aligned(v_pages, 15u) || !aligned(out, 15u) || !aligned(block_table, 3u) ||
        !aligned(cu_new, 3u) || !aligned(seq_lens, 3u) || !aligned(lse, 3u))
        return GQA_ERR_MISALIGNED;
    Call c;
    st = begin(c, q, cu_new, scale, out, lse, N, B, H, G, D, q_stride, workspace, workspace_bytes, stream);
    if (st != GQA_OK) return st;
    const long long slabs = (long long)num_pages * G;
    const int box = page_size < 128 ? page_size : 128;
    if ((st = encode_page_map(&c.a.tm_k, k_pages, slabs, page_size, D, box)) != GQA_OK) return st;
    if ((st = encode_page_map(&c.a.tm_v, v_pages, slabs, page_size, D, box)) != GQA_OK) return st;
    RaggedParams& p = c.a.p;
    p.lens = seq_lens;
    p.table = block_table;
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    return launch(c, D, true);
}

}  // extern "C"
