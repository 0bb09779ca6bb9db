// gqa_decode_paged_fp8: decode attention over a paged e4m3 cache.
//
// One CTA per query row: 128 keys a step, one thread per key for the score and
// one thread per column for the output, with the running maximum and sum of an
// online softmax.
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_decode.h"
#include "gqa_device.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

struct PagedFp8Params {
    const uint16_t* q;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* k_scale;
    const float* v_scale;
    const int32_t* table;
    const int32_t* lens;
    uint16_t* out;
    float* lse;
    float scale_log2;
    int B, sq, H, G, page_size, num_pages, max_pages, heads_per_group, blocks;
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    const uint32_t f = e4m3x2_to_f16x2(c);
    return __half2float(__ushort_as_half((unsigned short)f));
}

template <int D>
__global__ void __launch_bounds__(128) paged_fp8_kernel(const PagedFp8Params p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    __shared__ float q_s[D];
    __shared__ float w_s[128];
    __shared__ long long row_s[128];
    __shared__ float red[4];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int row = blockIdx.x;
    const int h = row % p.H, s = (row / p.H) % p.sq, b = row / p.H / p.sq;
    const int g = h / p.heads_per_group;
    const int T = clamp_len(p.lens[b], p.max_pages * p.page_size);
    const int n = T - p.sq + s + 1;                      // visible keys
    if (t < D) q_s[t] = __uint_as_float((uint32_t)p.q[(size_t)row * D + t] << 16);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int k0 = 0; k0 < n; k0 += 128) {
        __syncthreads();
        float x = -INFINITY, vs = 0.f;
        long long at = -1;
        if (k0 + t < n) {
            const int pos = k0 + t;
            const int page = p.table[(size_t)b * p.max_pages + pos / p.page_size];
            x = 0.f;
            if ((unsigned)page < (unsigned)p.num_pages) {
                const long long unit = (long long)page * p.G + g;
                at = (unit * p.page_size + pos % p.page_size) * D;
                const long long sc = unit * p.blocks + (pos % p.page_size) / 64;
                for (int d = 0; d < D; ++d) x += q_s[d] * e4m3_value(p.k_pages[at + d]);
                x *= p.k_scale[sc] * p.scale_log2;
                vs = p.v_scale[sc];
            }
        }
        float tile = x;
        for (int i = 16; i; i >>= 1) tile = fmaxf(tile, __shfl_xor_sync(0xffffffffu, tile, i));
        if (lane == 0) red[warp] = tile;
        __syncthreads();
        const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float pr = exp2f(x - ref);
        w_s[t] = pr * vs;
        row_s[t] = at;
        __syncthreads();
        float sum = pr;
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        if (lane == 0) red[warp] = sum;
        const float alpha = exp2f(m - ref);
        o *= alpha;
        if (t < D)
            for (int j = 0; j < 128 && k0 + j < n; ++j)
                if (row_s[j] >= 0) o += w_s[j] * e4m3_value(p.v_pages[row_s[j] + t]);
        __syncthreads();
        l = l * alpha + red[0] + red[1] + red[2] + red[3];
        m = m_new;
    }
    if (t < D) {
        const float y = l > 0.f || l != l ? o / l : 0.f;
        p.out[(size_t)row * D + t] = (uint16_t)(pack_bf16x2(y, 0.f) & 0xffffu);
    }
    if (p.lse && t == 0) p.lse[row] = l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace
}  // namespace gqa

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

}  // namespace

extern "C" {

size_t gqa_decode_paged_fp8_workspace_bytes(int B, int sq, int H, int G, int D, int page_size,
                                            int max_pages_per_seq) {
    if (check_paged_fp8(B, sq, H, G, D, page_size, max_pages_per_seq) != GQA_OK) return 0;
    return 256;
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
    const size_t need = gqa_decode_paged_fp8_workspace_bytes(B, sq, H, G, D, page_size, max_pages_per_seq);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return GQA_ERR_WORKSPACE;
    PagedFp8Params p;
    p.q = static_cast<const uint16_t*>(q);
    p.k_pages = static_cast<const uint8_t*>(k_pages);
    p.v_pages = static_cast<const uint8_t*>(v_pages);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = block_table;
    p.lens = seq_lens;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.B = B;
    p.sq = sq;
    p.H = H;
    p.G = G;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    p.heads_per_group = H / G;
    p.blocks = (page_size + 63) / 64;
    if (D == 64)
        paged_fp8_kernel<64><<<B * sq * H, 128, 0, stream>>>(p);
    else
        paged_fp8_kernel<128><<<B * sq * H, 128, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

}  // extern "C"
