// Attention of packed batches (gqa_prefill_packed, gqa_prefill_paged): a warp per
// query row, 32 keys at a time, one key per lane for the scores and D / 32 columns
// per lane for the product with V.
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_decode.h"
#include "gqa_device.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

struct RaggedParams {
    const uint16_t *q, *k, *v;
    uint16_t* out;
    float* lse;
    const int32_t *cu, *lens, *table;    // lens, table: paged only
    long long q_stride, k_stride, v_stride;
    float scale;
    int N, B, H, G, page_shift, num_pages, max_pages;
};

template <int D>
__global__ void __launch_bounds__(256) ragged_kernel(const RaggedParams p) {
    __shared__ float q_s[8][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + warp;
    pdl_launch_dependents();
    pdl_wait_primary();
    if (row >= (long long)p.N * p.H) return;
    const int n = (int)(row / p.H), h = (int)(row % p.H), g = h / (p.H / p.G);
    int b = 0;
    while (b < p.B && !(p.cu[b] <= n && n < p.cu[b + 1])) ++b;
    if (b == p.B) return;
    const int first = p.cu[b], end = min(p.cu[b + 1], p.N);
    const int T = p.table ? clamp_len(p.lens[b], p.max_pages << p.page_shift) : end - first;
    const int lim = T - end + n;
    for (int d = lane; d < D; d += 32)
        q_s[warp][d] = __uint_as_float((uint32_t)p.q[n * p.q_stride + h * D + d] << 16) * (p.scale * 1.4426950408889634f);
    __syncwarp();
    auto key = [&](int t) -> long long {      // element of position t's row in k and v, -1: reads as zeros
        if (!p.table) return -2;
        const int page = p.table[(size_t)b * p.max_pages + (t >> p.page_shift)];
        if ((unsigned)page >= (unsigned)p.num_pages) return -1;
        return ((((long long)page * p.G + g) << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * D;
    };
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int t0 = 0; t0 <= lim; t0 += 32) {
        const int t = t0 + lane;
        const bool see = t <= lim;
        const long long at = see ? key(t) : -1;
        float x = see ? 0.f : -INFINITY;
        if (see && at != -1) {
            const uint16_t* k = p.table ? p.k + at : p.k + (first + t) * p.k_stride + g * D;
            for (int d = 0; d < D; ++d) x = fmaf(__uint_as_float((uint32_t)k[d] << 16), q_s[warp][d], x);
        }
        float top = x;
        for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
        const float a = exp2f(m - base), e = see ? exp2f(x - base) : 0.f;
        l = l * a + e;
        m = mn;
        for (int i = 0; i < D / 32; ++i) o[i] *= a;
        for (int j = 0; j < 32 && t0 + j <= lim; ++j) {
            const float pj = __shfl_sync(0xffffffffu, e, j);
            const long long vj = __shfl_sync(0xffffffffu, at, j);
            if (vj == -1) continue;
            const uint16_t* v = p.table ? p.v + vj : p.v + (first + t0 + j) * p.v_stride + g * D;
            for (int i = 0; i < D / 32; ++i)
                o[i] = fmaf(pj, __uint_as_float((uint32_t)v[i * 32 + lane] << 16), o[i]);
        }
    }
    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    for (int i = 0; i < D / 32; ++i)
        p.out[row * D + i * 32 + lane] = (uint16_t)pack_bf16x2(l == 0.f ? 0.f : o[i] / l, 0.f);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

bool aligned(const void* x, unsigned mask) { return (reinterpret_cast<uintptr_t>(x) & mask) == 0; }

int check_sizes(int N, int B, int H, int G, int D) {
    if (N < 0 || B <= 0 || H <= 0 || G <= 0 || D <= 0) return GQA_ERR_INVALID_ARG;
    if (H % G != 0) return GQA_ERR_HEAD_RATIO;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (H / G > 128 || (long long)N * H >= (1ll << 31) || B >= (1 << 24) || G >= (1 << 20)) return GQA_ERR_UNSUPPORTED;
    return GQA_OK;
}

int check_rows(const void* x, long long stride, int heads, int D) {
    if (stride < (long long)heads * D) return GQA_ERR_INVALID_ARG;
    if (!aligned(x, 15u) || (stride & 7)) return GQA_ERR_MISALIGNED;
    return stride >= (1ll << 38) ? GQA_ERR_UNSUPPORTED : GQA_OK;
}

size_t workspace_need(int N, int B, int H, int G, int D, int sms) { return 256; }

int launch(RaggedParams& p, int D, cudaStream_t stream) {
    const long long rows = (long long)p.N * p.H;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (D == 64)
        ragged_kernel<64><<<grid, 256, 0, stream>>>(p);
    else
        ragged_kernel<128><<<grid, 256, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
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
    return workspace_need(N, B, H, G, D, sms);
}

int gqa_prefill_packed(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, float scale,
                       void* out, float* lse, int N, int B, int H, int G, int D, long long q_stride,
                       long long k_stride, long long v_stride, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    int st = check_sizes(N, B, H, G, D);
    if (st != GQA_OK) return st;
    if (N == 0) return GQA_OK;              // tensors without rows have no address
    if (!q || !k || !v || !cu_seqlens || !out || !(scale > 0.f) || scale > 3.0e38f) return GQA_ERR_INVALID_ARG;
    if ((st = check_rows(q, q_stride, H, D)) != GQA_OK || (st = check_rows(k, k_stride, G, D)) != GQA_OK ||
        (st = check_rows(v, v_stride, G, D)) != GQA_OK)
        return st;
    if (!aligned(out, 15u) || !aligned(cu_seqlens, 3u) || !aligned(lse, 3u)) return GQA_ERR_MISALIGNED;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    if (!workspace || workspace_bytes < workspace_need(N, B, H, G, D, sms) || !aligned(workspace, 255u))
        return GQA_ERR_WORKSPACE;
    RaggedParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.cu = cu_seqlens;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.scale = scale;
    p.N = N;
    p.B = B;
    p.H = H;
    p.G = G;
    return launch(p, D, stream);
}

int gqa_prefill_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                      const int32_t* cu_new, const int32_t* seq_lens, float scale, void* out, float* lse, int N,
                      int B, int H, int G, int D, long long q_stride, int page_size, int num_pages,
                      int max_pages_per_seq, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check_sizes(N, B, H, G, D);
    if (st != GQA_OK) return st;
    if (N == 0) return GQA_OK;              // tensors without rows have no address
    if (!q || !k_pages || !v_pages || !block_table || !cu_new || !seq_lens || !out || !(scale > 0.f) || scale > 3.0e38f ||
        page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0)
        return GQA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1))) return GQA_ERR_UNSUPPORTED;
    if ((long long)max_pages_per_seq * page_size >= (1ll << 31) - 128 || (long long)num_pages * G >= (1ll << 31) - 1)
        return GQA_ERR_UNSUPPORTED;
    if ((st = check_rows(q, q_stride, H, D)) != GQA_OK) return st;
    if (!aligned(k_pages, 15u) || !aligned(v_pages, 15u) || !aligned(out, 15u) || !aligned(block_table, 3u) ||
        !aligned(cu_new, 3u) || !aligned(seq_lens, 3u) || !aligned(lse, 3u))
        return GQA_ERR_MISALIGNED;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    if (!workspace || workspace_bytes < workspace_need(N, B, H, G, D, sms) || !aligned(workspace, 255u))
        return GQA_ERR_WORKSPACE;
    RaggedParams p = {};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_pages);
    p.v = static_cast<const uint16_t*>(v_pages);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.cu = cu_new;
    p.lens = seq_lens;
    p.table = block_table;
    p.q_stride = q_stride;
    p.scale = scale;
    p.N = N;
    p.B = B;
    p.H = H;
    p.G = G;
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    return launch(p, D, stream);
}

}  // extern "C"
