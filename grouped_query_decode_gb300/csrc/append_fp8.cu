// gqa_append_paged_fp8: the new tokens' K/V, quantised into a paged e4m3 cache.
//
// One group of threads per (sequence, block of tokens, KV head, K or V):
//   top    = max |x| over the block's finite new elements
//   scale' = the block's scale, if it holds earlier tokens and top <= 448 scale;
//            else the smallest 2^e >= top / 448
//   codes  = e4m3(x / scale'); kept codes = e4m3(code * (scale / scale')) if it moved
// The new elements are read once, into registers, where they wait for the
// maximum. Nothing is shared between groups, so no order of execution changes
// a result.
//
// Bytes: 2 read and 1 written per element. Four threads a token of a block, a run
// of blocks each, the next block's tokens under way behind the present one's
// maximum and conversion: 2048 tokens of four sequences, 8 KV heads of 128 (50
// MB), 11.0 us, 4.6 TB/s with the launch's 2 us (8 x 8192 tokens 65 us, 6.2
// TB/s). The schedulers issue 60 % of the time there, so instructions count: two
// products to an instruction, packed maxima, no division by the page size (13.4
// us without these). Up to 8 new tokens a warp takes a block by itself: one token of 64
// sequences 2.4 us, which is latency (length, then page and tokens, then codes);
// of the 64 registers that leaves a thread at D 128, 28 bytes are spilled.
#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_decode.h"
#include "gqa_device.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kBlockTokens = 64;   // most tokens that share a scale

struct AppendParams {
    const uint16_t* x_new[2];   // K, V: [B, sq, G, D] bf16
    uint8_t* pages[2];          // [num_pages, G, page_size, D] codes
    float* scale[2];            // [num_pages, G, blocks of a page]
    const int32_t* table;
    const int32_t* lens;
    int B, sq, G, page_size, num_pages, max_pages;
    int page_shift;             // log2 of page_size
    int size, size_shift;       // tokens of a block: min(64, page_size)
    int blocks;                 // blocks of a sequence that may receive tokens
    int per, runs;              // blocks per item, items per sequence and head
};

// Smallest power of two >= top / 448 (448 = 0.875 * 2^9), 0 for 0, at least 2^-126.
__device__ __forceinline__ float scale_for(float top) {
    if (top == 0.f) return 0.f;
    const uint32_t bits = __float_as_uint(top);
    int e = (int)(bits >> 23) - 126;                     // top = m * 2^e, m in [0.5, 1)
    e += (bits & 0x7fffffu) > 0x600000u ? -8 : -9;       // m > 0.875
    if ((bits >> 23) == 0 || e < -126) e = -126;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// x / scale; for a power of two by its reciprocal, which is as exact.
struct Divider {
    float scale, inv;
    bool pow2;
    __device__ explicit Divider(float s) : scale(s) {
        const uint32_t b = __float_as_uint(s);
        pow2 = (b & 0x7fffffu) == 0 && (b >> 23) != 0 && (b >> 23) < 254;
        inv = pow2 ? __uint_as_float((254u - (b >> 23)) << 23) : 0.f;   // 2^-e
    }
    // A scale of 0 comes with zeros and with NaN, which stays.
    __device__ float operator()(float x) const { return pow2 ? x * inv : (scale == 0.f ? x * 0.f : __fdiv_rn(x, scale)); }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float finite_or_nan(float x) {
    return fabsf(x) <= 3.4028234664e38f ? x : __uint_as_float(0x7fffffffu);
}

// e4m3 codes of two bf16 values times f, both products in one instruction.
__device__ __forceinline__ uint32_t scaled_codes(uint32_t w, float f) {
    unsigned long long x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(w << 16), "r"(w & 0xffff0000u));
    asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(f));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
    return e4m3x2(lo, hi);
}

// Eight bf16 values.
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// TPI threads (a warp, or the CTA) per item; an item is a run of `per` blocks of
// one (sequence, KV head, K or V). CHUNKS: 8-element chunks of a block's new
// tokens per thread at most. A block's tokens are on their way while the one
// before is quantised; what a block needs first (length, then page and tokens)
// is two reads deep.
template <int D, int TPI, int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) append_kernel(const __grid_constant__ AppendParams p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    constexpr int kRowChunks = D / 8;
    const int t = threadIdx.x % TPI;
    const unsigned item = blockIdx.x * (THREADS / TPI) + threadIdx.x / TPI;
    const unsigned heads = 2u * p.G;
    if (item >= heads * p.runs * p.B) return;        // whole groups leave
    const unsigned rest = item / heads, head = item - rest * heads;
    const int which = head & 1, g = head >> 1;
    const int b = rest / p.runs, run = rest - b * p.runs;
    const int T = clamp_len(p.lens[b], p.max_pages * p.page_size);
    const int begin = T > p.sq ? T - p.sq : 0;       // first position that gets a new token
    const int begin_block = begin >> p.size_shift;
    const int block0 = begin_block + run * p.per;
    const int block1 = min(block0 + p.per, min((T + p.size - 1) >> p.size_shift, begin_block + p.blocks));
    const int shift = T - p.sq;                      // new token s sits at position shift + s
    const uint16_t* x = p.x_new[which] + ((size_t)b * p.sq * p.G + g) * D;
    const size_t row_step = (size_t)p.G * D;
    // This thread's chunks of a block: one column, every TPI / kRowChunks rows.
    static_assert(TPI % kRowChunks == 0, "whole rows");
    x += (t / kRowChunks) * row_step + (t % kRowChunks) * 8;
    const size_t chunk_step = (TPI / kRowChunks) * row_step;
    const int page_blocks = (p.page_size + kBlockTokens - 1) / kBlockTokens;
    const int32_t* table = p.table + (size_t)b * p.max_pages;

    // The tokens and the page of a block.
    uint4 next[CHUNKS];
    int next_page = -1;
    auto load = [&](int block) {
        const int start = block * p.size;
        const int lo = max(begin, start), hi = min(T, start + p.size);
        next_page = table[start >> p.page_shift];
        const uint16_t* x0 = x + (size_t)(lo - shift) * row_step;
        const int n = (hi - lo) * kRowChunks;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const int i = t + c * TPI;
            next[c] = make_uint4(0, 0, 0, 0);
            if (i < n)
                next[c] = *reinterpret_cast<const uint4*>(x0 + c * chunk_step);
        }
    };
    // Largest value of the group; every thread of it has passed its reads then.
    int turn = 0;
    auto group_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (TPI > 32) {
            __shared__ __align__(16) uint32_t part[2][TPI / 32];
            uint32_t* mine = part[turn];             // the other half may still be read
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < TPI / 32; w += 2) {
                const uint2 u = *reinterpret_cast<const uint2*>(mine + w);
                m = max(m, max(u.x, u.y));
            }
        } else {
            __syncwarp();
        }
        return m;
    };
    if (block0 < block1) load(block0);
    for (int block = block0; block < block1; ++block) {
        uint4 v[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) v[c] = next[c];
        const int page = next_page;
        if (block + 1 < block1) load(block + 1);
        if ((unsigned)page >= (unsigned)p.num_pages) continue;       // the whole group goes on
        const int start = block * p.size;
        const int lo = max(begin, start), hi = min(T, start + p.size);
        const int kept = lo - start, n = (hi - lo) * kRowChunks;
        const int in_page = start & (p.page_size - 1);
        const size_t unit = (size_t)page * p.G + g;
        uint8_t* rows = p.pages[which] + (unit * p.page_size + in_page) * D;
        float* scale_at =
            p.scale[which] + unit * page_blocks + in_page / kBlockTokens;
        const float held = kept > 0 ? *scale_at : 0.f;
        // Magnitudes order as their bits do, two at a time. Infinities and NaN
        // do not count; blocks with one are rare and read their tokens again.
        uint32_t m2 = 0;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            m2 = __vmaxu2(m2, __vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu));
            m2 = __vmaxu2(m2, __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu));
        }
        const uint16_t* x0 = x + (size_t)(lo - shift) * row_step;
        auto chunk_at = [&](int i) {             // i: t, t + TPI, ...
            return *reinterpret_cast<const uint4*>(x0 + (i / TPI) * chunk_step);
        };
        uint32_t m = group_max(max(m2 & 0xffffu, m2 >> 16));
        const bool odd = m >= 0x7f80u;
        if (odd) {
            m = 0;
#pragma unroll 1
            for (int i = t; i < n; i += TPI) {
                const uint4 u = chunk_at(i);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t hi16 = (w[k] >> 16) & 0x7fffu, lo16 = w[k] & 0x7fffu;
                    m = max(m, max(hi16 < 0x7f80u ? hi16 : 0u, lo16 < 0x7f80u ? lo16 : 0u));
                }
            }
            m = group_max(m);
        }
        const float top = __uint_as_float(m << 16);
        const float old = held > 0.f ? held : 0.f;
        const float scale = old > 0.f && top <= kE4m3Max * old ? old : scale_for(top);
        const Divider div(scale);
        if (div.pow2 && !odd) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const int i = t + c * TPI;
                if (i < n) {
                    uint2 w;
                    w.x = scaled_codes(v[c].x, div.inv) | (scaled_codes(v[c].y, div.inv) << 16);
                    w.y = scaled_codes(v[c].z, div.inv) | (scaled_codes(v[c].w, div.inv) << 16);
                    *reinterpret_cast<uint2*>(rows + (size_t)kept * D + (size_t)i * 8) = w;
                }
            }
        } else {
#pragma unroll 1
            for (int i = t; i < n; i += TPI) {
                float x8[8];
                unpack8(chunk_at(i), x8);
#pragma unroll
                for (int e = 0; e < 8; ++e) x8[e] = div(finite_or_nan(x8[e]));
                uint2 w;
                w.x = e4m3x2(x8[0], x8[1]) | (e4m3x2(x8[2], x8[3]) << 16);
                w.y = e4m3x2(x8[4], x8[5]) | (e4m3x2(x8[6], x8[7]) << 16);
                *reinterpret_cast<uint2*>(rows + (size_t)kept * D + (size_t)i * 8) = w;
            }
        }
        if (kept > 0 && scale != old) {
            const float r = scale > 0.f ? __fdiv_rn(old, scale) : 0.f;
            for (int i = t; i < kept * (D / 16); i += TPI) {
                uint4* at = reinterpret_cast<uint4*>(rows) + i;
                const uint4 c = *at;
                const uint32_t in[4] = {c.x, c.y, c.z, c.w};
                uint32_t out[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t y = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t f = e4m3x2_to_f16x2((uint16_t)(in[q] >> (16 * h)));
                        const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&f));
                        y |= e4m3x2(f2.x * r, f2.y * r) << (16 * h);
                    }
                    out[q] = y;
                }
                *at = make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
        if (t == 0) *scale_at = scale;
    }
}

template <int D, int TPI, int THREADS, int CHUNKS>
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
    const long long items = 2ll * p.G * p.runs * p.B;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items + THREADS / TPI - 1) / (THREADS / TPI)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel<D, TPI, THREADS, CHUNKS>, p);
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_append_paged_fp8(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                                    float* k_scale, float* v_scale, const int32_t* block_table,
                                    const int32_t* seq_lens, int B, int sq, int G, int D, int page_size,
                                    int num_pages, int max_pages_per_seq, cudaStream_t stream) {
    if (B <= 0 || sq <= 0 || G <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0)
        return GQA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1))) return GQA_ERR_UNSUPPORTED;
    if (!k_new || !v_new || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !seq_lens)
        return GQA_ERR_INVALID_ARG;
    const uintptr_t wide = reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
                           reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages);
    const uintptr_t word = reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
                           reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens);
    if ((wide & 15u) || (word & 3u)) return GQA_ERR_MISALIGNED;
    AppendParams p;
    p.x_new[0] = static_cast<const uint16_t*>(k_new);
    p.x_new[1] = static_cast<const uint16_t*>(v_new);
    p.pages[0] = static_cast<uint8_t*>(k_pages);
    p.pages[1] = static_cast<uint8_t*>(v_pages);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.table = block_table;
    p.lens = seq_lens;
    p.B = B;
    p.sq = sq;
    p.G = G;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    p.size = page_size < kBlockTokens ? page_size : kBlockTokens;
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.size_shift = __builtin_ctz((unsigned)p.size);
    p.blocks = (int)(((long long)sq + p.size - 2) / p.size) + 1;
    if ((long long)max_pages_per_seq * page_size >= (1ll << 31) - kBlockTokens || sq >= (1 << 30) ||
        2ll * G * p.blocks * B >= (1ll << 31))
        return GQA_ERR_UNSUPPORTED;
    // Up to 8 new tokens a sequence: a warp per block holds them in registers;
    // beyond that a CTA of four threads per token of a block does, 1024 threads to
    // an SM, with a run of blocks (4 x 2048 tokens in 16-token pages: 23.5 us with
    // 256 threads a block, 11.0 with 64; 32-token pages 16.0 and 10.9).
    int sms;
    unsigned* status;
    const int st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    p.per = 1;
    if (sq > 8) {
        // The run that ends first: a block's time each, half of one to start, and
        // the CTAs beyond those that are resident at once take turns, half a run
        // of which the others wait for. Runs of 1 | 2 | 3 | 4 | 6 blocks, us: 4 x 2048
        // tokens 12.2 | 11.9 | 12.4 | 11.0 | 14.1; 3 x 777 4.0 | 5.1 | 6.5 | | 9.7; 8 x
        // 8192 72.9 | 68.3 | 66.1 | | 64.8 (as few as fit at once, 28: 76.7).
        const long long slots = 1024ll / (4 * p.size) * sms;
        long long best = 0;
        for (int per = 1; per <= 8; ++per) {
            const long long ctas = 2ll * G * B * ((p.blocks + per - 1) / per);
            const long long cost = ctas <= slots ? (2 * per + 1) * slots : ctas * (2 * per + 1) + per * slots;
            if (best == 0 || cost < best) {
                best = cost;
                p.per = per;
            }
        }
    }
    if (p.per > p.blocks) p.per = p.blocks;
    p.runs = (p.blocks + p.per - 1) / p.per;
    cudaError_t e;
    if (sq <= 8)
        e = D == 64 ? launch_append<64, 32, 128, 2>(p, stream) : launch_append<128, 32, 128, 4>(p, stream);
    else if (p.size == 16)
        e = D == 64 ? launch_append<64, 64, 64, 2>(p, stream) : launch_append<128, 64, 64, 4>(p, stream);
    else if (p.size == 32)
        e = D == 64 ? launch_append<64, 128, 128, 2>(p, stream) : launch_append<128, 128, 128, 4>(p, stream);
    else
        e = D == 64 ? launch_append<64, 256, 256, 2>(p, stream) : launch_append<128, 256, 256, 4>(p, stream);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}
