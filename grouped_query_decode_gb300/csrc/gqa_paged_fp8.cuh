// Decode attention over a paged e4m3 cache on the 5th-generation tensor cores,
// with the codes as operands: no K or V element is converted.
//
// A unit is (sequence, KV head, up to 32 query rows). Its keys are cut into
// 128-token tiles; tokens sit on the products' M side, rows on the N side:
//     S [128 tokens x 2 rows]  = K   [128 x D]   (smem, K-major)  x Q^T  (smem)
//     O [D x 4 rows]          += V^T [D x 128]   (smem, MN-major) x P    (smem)
// both kind::f8f6f4 with fp32 accumulators in tensor memory. Rows are few, so
// each bf16 or fp16 number on the N side is spread over several 8-bit columns:
//   q * 2^e = hi + lo / 16, e4m3 (2^e brings the row's maximum to [128, 256)):
//     4 significant bits each, the residual an exact difference, so every bf16
//     query down to 2^-13 of its row's maximum, and 2^-21 of it below that;
//   w = fp16(p * v_scale * 2^c) = t0 + t1 + t2 + t3, e5m2: a term is the upper
//     byte of the fp16 residual (its first 3 significant bits), the next
//     residual the exact difference, so 4 terms are all 11 bits of w down to
//     2^-6, and w within 2^-16 below that, where w is 1024..2048 for p = 1. No
//     conversion instruction is needed; an e4m3 split takes two per term and
//     pair, and those, at a quarter of the rate, took half of a tile's time.
// The extra columns cost nothing: up to N = 128 a product of M = 128 takes the
// 64 cycles that reading its K or V rows takes.
//
// Softmax, one thread per token: x = s * scale2 * k_scale (base 2), p = 2^(x - m)
// with a reference m per row that moves only when a score exceeds it by more
// than 2 (then O is rescaled in tensor memory), so that tiles need no maximum
// across threads: one vote. The sum l is kept per thread until the end. v_scale enters
// p through a power of two 2^c that follows the largest scale seen.
//
// Work: the tiles of all units, end to end, are shared equally by the CTAs
// (one per SM); a unit that crosses CTAs leaves (O, m, l) per CTA in the
// workspace for the merge kernel. Per CTA: two groups of four softmax warps
// take alternate tiles, two warps bring K and V by TMA (a box per page, the
// swizzle of the operand layout), one issues the products, one prepares Q.
// Every wait is bounded, as in the other kernels.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "gqa_device.cuh"
#include "gqa_paged_fp8.h"
#include "tcgen05.cuh"

namespace gqa {

constexpr int kP8Threads = 384;
constexpr int kP8Terms = 4;               // e5m2 columns per probability
constexpr float kP8Slack = 4.0f;          // p <= 2^4 before the reference moves
constexpr float kP8ProbScale = 2048.0f;   // p * v_scale * 2^-ev * 2048 <= 16 * 1.75 * 2048 = 57344
constexpr float kP8ScaleSlack = 1.75f;
constexpr float kP8Unseen = -3.402823466e38f;   // reference of a row that has seen no key

template <int D, int RP>
struct P8Shape {
    static constexpr int kTileBytes = kP8Tokens * D;              // K or V of one tile
    static constexpr int kNs = 2 * RP;                            // columns of S: hi, lo
    static constexpr int kNp = kP8Terms * RP;                     // columns of O
    static constexpr int kQBytes = kNs * D;
    static constexpr int kPBytes = kP8Tokens * kNp;
    // The rings take what the rest leaves of 227 KB. A V tile is held from its
    // copy to P V, a K tile only to S, so V gets more stages.
    static constexpr int kStagesK = (D == 128 ? 1 : 2) * (RP == 32 ? 4 : 5);
    static constexpr int kStagesV = (D == 128 ? 1 : 2) * (RP == 32 ? 5 : 7);
    static constexpr int kBars = 2 * (kStagesK + kStagesV) + 15;
    static constexpr int kRowInfoBytes = 2 * 3 * RP * 4;
    static constexpr int kRefBytes = 2 * RP * 4;
    static constexpr int kWarpMaxBytes = 2 * 4 * (RP + 1) * 4;
    static constexpr int kSumBytes = 2 * RP * 16;
    static constexpr int kMergeBytes = 3 * RP * 8;                // group 1's (m, l); each group's row factors
    static constexpr int kLenBytes = kP8Threads * 4;
    static constexpr int kMiscBytes = 192;
    static constexpr int kSmemBytes = 1024 + (kStagesK + kStagesV) * kTileBytes + 2 * kQBytes + 2 * kPBytes +
                                      kRowInfoBytes + kRefBytes + kWarpMaxBytes + kSumBytes + kMergeBytes +
                                      kLenBytes + kMiscBytes + 8 * kBars;
    // Group 1 hands its O over in its own P operand, which its last product has read.
    static_assert(RP * D * 4 <= kPBytes, "O fits P");
    static constexpr uint32_t kColS = 0, kColO = 2 * kNs;         // S_0 | S_1 | O_0 | O_1
    static constexpr uint32_t kCols = 2 * kNs + 2 * kNp;
    static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
};

// ------------------------------------------------------ tensor-core wrappers

// Shared-memory matrix descriptor: as smem_desc_sw128, with the layout given
// (2: 128-byte swizzle, 4: 64-byte swizzle, 0: none).
__device__ __forceinline__ uint64_t p8_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t layout) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (layout << 61);
}

// Instruction descriptor of kind::f8f6f4: e4m3 A, e4m3 or e5m2 B, fp32 accumulator.
__host__ __device__ constexpr uint32_t p8_idesc(int M, int N, bool a_mn, bool b_mn, bool b_e5m2) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 fp32 columns of this thread's TMEM lane, waited on; and their store.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ------------------------------------------------------------ e4m3 and fp16

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// What is left of two fp16 values without their first e5m2 terms (exact).
__device__ __forceinline__ uint32_t e5m2_residual(uint32_t f) {
    const uint32_t t = f & 0xff00ff00u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&f), *reinterpret_cast<const __half2*>(&t));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// Floats to integers of the same order, and back.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // |e| <= 126

// ---------------------------------------------------------------------- plan

// Lengths, from the CTA's copy where the batch fits it, and the tiles that the
// rows of an entry (b, row tile) see: with one row tile, all of the sequence's.
template <int RP>
struct P8Lens {
    const PagedFp8Params& p;
    const int* copy;
    __device__ int global(int b) const { return clamp_len(p.lens[b], p.max_pages << p.page_shift); }
    __device__ int tokens(int b) const { return p.B <= kP8Threads ? copy[b] : global(b); }
    __device__ void split(int entry, int& b, int& rt) const {
        b = p.row_tiles == 1 ? entry : entry / p.row_tiles;
        rt = entry - b * p.row_tiles;
    }
    __device__ int tiles(int entry) const {
        int b, rt;
        split(entry, b, rt);
        const int T = tokens(b);
        if (p.row_tiles == 1) return (T + kP8Tokens - 1) / kP8Tokens;
        const int last = min(p.R, (rt + 1) * RP) - 1;
        const int lim = T - p.sq + last / p.heads_per_group;
        return lim < 0 ? 0 : lim / kP8Tokens + 1;
    }
};

// A CTA's share as a run of segments of units.
struct P8Segment {
    int entry, g, i0, i1, n;     // tiles [i0, i1) of the unit's n
};
template <int RP>
struct P8Walk {
    long long left;
    int entry, g, off;
    __device__ bool next(const P8Lens<RP>& lens, P8Segment& s) {
        if (left <= 0) return false;
        int n = lens.tiles(entry);
        while (n == 0) n = lens.tiles(++entry);
        s.entry = entry;
        s.g = g;
        s.i0 = off;
        s.i1 = left < n - off ? off + (int)left : n;
        s.n = n;
        left -= s.i1 - s.i0;
        off = 0;
        if (++g == lens.p.G) {
            g = 0;
            ++entry;
        }
        return true;
    }
};

struct P8Plan {
    long long total, begin, end;   // tiles of the call, and this CTA's
    int entry, g, off;             // where it begins
    int ctas;                      // CTAs that share the tiles
};

// a * b / c for 64-bit a, in 32 bits where they do.
__device__ __forceinline__ long long muldiv(long long a, int b, int c) {
    const unsigned long long x = (unsigned long long)a * (unsigned)b;
    return x >> 32 ? (long long)(x / (unsigned)c) : (long long)((unsigned)x / (unsigned)c);
}

// All threads: sums the tiles of all entries, each thread over a contiguous
// range of them, and finds where this CTA's share begins. The caller
// synchronises the CTA before anyone reads the plan.
template <int RP>
__device__ void p8_make_plan(const P8Lens<RP>& lens, int* len_copy, P8Plan* plan, long long* warp_sum) {
    const PagedFp8Params& p = lens.p;
    const int entries = p.B * p.row_tiles;
    const int per = (entries + kP8Threads - 1) / kP8Threads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.B <= kP8Threads && p.row_tiles > 1) {
        if ((int)threadIdx.x < p.B) len_copy[threadIdx.x] = lens.global(threadIdx.x);
        __syncthreads();
    } else if ((int)threadIdx.x < p.B && p.B <= kP8Threads) {
        len_copy[threadIdx.x] = lens.global(threadIdx.x);    // read back below by this thread only
    }
    const int e0 = (int)min((long long)entries, (long long)threadIdx.x * per), e1 = min(entries, e0 + per);
    long long mine = 0;
    for (int e = e0; e < e1; ++e) mine += lens.tiles(e);
    mine *= p.G;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    long long before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kP8Threads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    const long long most = total / kP8MinTiles;
    const int ctas = most < 1 ? 1 : most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
    const int c = blockIdx.x;
    const long long t0 = c < ctas ? muldiv(total, c, ctas) : total;
    const long long t1 = c < ctas ? muldiv(total, c + 1, ctas) : total;
    if (t0 < t1 ? t0 >= before && t0 < before + mine : threadIdx.x == 0) {
        plan->total = total;
        plan->begin = t0;
        plan->end = t1;
        plan->ctas = ctas;
        plan->entry = plan->g = plan->off = 0;
        if (t0 < t1) {
            long long at = before;
            int e = e0, n = lens.tiles(e);
            while (at + (long long)n * p.G <= t0) {
                at += (long long)n * p.G;
                n = lens.tiles(++e);
            }
            const unsigned in = (unsigned)min(t0 - at, 0xffffffffll);   // below n * G
            plan->entry = e;
            plan->g = t0 - at > 0xffffffffll ? (int)((t0 - at) / n) : (int)(in / (unsigned)n);
            plan->off = (int)(t0 - at - (long long)plan->g * n);
        }
    }
}

// Sums v[r] of the warp's lanes; lane i returns row i % RP. v is overwritten.
template <int RP>
__device__ __forceinline__ float reduce_rows(float (&v)[RP], int lane) {
#pragma unroll
    for (int o = RP / 2; o >= 1; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o];
            const float keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float s = v[0];
#pragma unroll
    for (int o = RP; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Query row r of entry (b, rt): its index in [B, sq, H], or -1 past the last.
template <int RP>
__device__ __forceinline__ int p8_out_row(const PagedFp8Params& p, int b, int rt, int g, int r, int* s_tok) {
    const int rr = rt * RP + r;
    if (rr >= p.R) return -1;
    const int s = rr / p.heads_per_group;
    *s_tok = s;
    return (b * p.sq + s) * p.H + g * p.heads_per_group + (rr - s * p.heads_per_group);
}

// ------------------------------------------------------------------- kernel

// A group's 128 threads meet (and agree whether any of them votes). These are
// the CTA's named barriers 1 and 2: no thread of a group ever leaves its loop
// early, whatever a bounded wait reported, so the four warps always arrive.
__device__ __forceinline__ void group_sync(int x) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(x + 1) : "memory"); }
__device__ __forceinline__ bool group_any(int x, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(x + 1)
        : "memory");
    return r != 0;
}

template <int D, int RP>
__global__ void __launch_bounds__(kP8Threads, 1)
    gqa_paged_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const PagedFp8Params p) {
    using PS = P8Shape<D, RP>;
    constexpr int SK = PS::kStagesK, SV = PS::kStagesV;
    constexpr uint32_t TB = PS::kTileBytes;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t k_s = base, v_s = k_s + SK * TB, q_s = v_s + SV * TB, p_s = q_s + 2 * PS::kQBytes;
    unsigned char* gen = smem_raw + (p_s + 2 * PS::kPBytes - raw);
    float* stage_o = reinterpret_cast<float*>(gen - PS::kPBytes);         // [RP][D], in group 1's P
    // Rows of the unit in q buffer i: scale2 * 2^-e, last visible key, output row.
    float* row_scale = reinterpret_cast<float*>(gen);                     // [2][RP]
    int* row_lim = reinterpret_cast<int*>(row_scale + 2 * RP);            // [2][RP]
    int* row_out = row_lim + 2 * RP;                                      // [2][RP]
    gen += PS::kRowInfoBytes;
    float4* sums = reinterpret_cast<float4*>(gen);                        // [2][RP], one component a warp
    gen += PS::kSumBytes;
    float* neg_ref = reinterpret_cast<float*>(gen);                       // [2][RP]: -m
    gen += PS::kRefBytes;
    float2* other = reinterpret_cast<float2*>(gen);                       // [RP]: (m, l) of group 1
    float2* factors = other + RP;                                         // [2][RP]: weights of the groups' O
    gen += PS::kMergeBytes;
    int* warp_max = reinterpret_cast<int*>(gen);                          // [2][4][RP + 1]
    gen += PS::kWarpMaxBytes;
    int* len_copy = reinterpret_cast<int*>(gen);
    gen += PS::kLenBytes;
    P8Plan* plan = reinterpret_cast<P8Plan*>(gen);                        // 40 bytes
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + 64);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gen + 68);
    long long* warp_sum = reinterpret_cast<long long*>(gen + 80);         // [12]
    gen += PS::kMiscBytes;
    const uint32_t bar0 = smem_addr(gen);
    const uint32_t k_full = bar0, k_empty = k_full + 8 * SK, v_full = k_empty + 8 * SK, v_empty = v_full + 8 * SV;
    const uint32_t q_full = v_empty + 8 * SV, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, s_free = s_full + 16, p_full = s_free + 16;
    const uint32_t m_full = p_full + 16, m_empty = m_full + 8, fin = m_empty + 8;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = p.wait_timeout_ns;
    const P8Lens<RP> lens = {p, len_copy};

    if (threadIdx.x == 0) {
        for (int s = 0; s < SK; ++s) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
        }
        for (int s = 0; s < SV; ++s) {
            mbar_init(v_full + 8 * s, 1);
            mbar_init(v_empty + 8 * s, 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(q_full + 8 * x, 1);
            mbar_init(q_empty + 8 * x, 9);     // eight softmax warps and the products
            mbar_init(s_full + 8 * x, 1);
            mbar_init(s_free + 8 * x, 4);
            mbar_init(p_full + 8 * x, 4);
            mbar_init(fin + 8 * x, 1);
        }
        mbar_init(m_full, 4);
        mbar_init(m_empty, 4);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_addr(tmem_slot), PS::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 8 && lane < 2) tma_prefetch_desc(lane ? &tm_v : &tm_k);
    tc_fence_before();
    pdl_launch_dependents();
    pdl_wait_primary();
    p8_make_plan<RP>(lens, len_copy, plan, warp_sum);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    P8Walk<RP> walk = {plan->end - plan->begin, plan->entry, plan->g, plan->off};
    P8Segment seg;
    // Bounded waits of one thread, and of a softmax warp: all its lanes poll,
    // and all go on when the limit runs out.
    auto wait = [&](uint32_t bar, uint32_t n) { return wait_phase(bar, n & 1, abort_flag, p.status, tmo); };
    auto all_wait = [&](uint32_t bar, uint32_t n) {
        if (!mbar_try_wait(bar, n & 1) && !*abort_flag) wait_phase(bar, n & 1, abort_flag, p.status, tmo);
        __syncwarp();
    };

    if (warp == 8) {
        // ------------------------------------- loader: lanes 0-7 K, lanes 8-15 V
        const bool is_v = lane >= 8;
        const int box_of = lane & 7;
        const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
        const uint32_t full = is_v ? v_full : k_full, empty = is_v ? v_empty : k_empty;
        const uint32_t ring = is_v ? v_s : k_s;
        const int S = is_v ? SV : SK;
        const int page_size = 1 << p.page_shift;
        const int box = min(page_size, kP8Tokens);
        const int boxes = kP8Tokens / box;
        const uint64_t pol = l2_policy_evict_first();
        int it = 0, issued = 0, s = 0;
        uint32_t ph = 1;
        bool ok = true;
        while (ok && walk.next(lens, seg)) {
            int b, rt;
            lens.split(seg.entry, b, rt);
            const int T = lens.tokens(b);
            const int32_t* row = p.table + (size_t)b * p.max_pages;
            // This lane's page of a tile; looked up one tile ahead.
            auto lookup = [&](int i) {
                const int pos = i * kP8Tokens + box_of * box;
                return lane < 16 && box_of < boxes && i < seg.i1 && pos < T ? row[pos >> p.page_shift] : -1;
            };
            int page = lookup(seg.i0);
            for (int i = seg.i0; i < seg.i1; ++i, ++it) {
                const int cur = page;
                page = lookup(i + 1);
                const int pos = i * kP8Tokens + box_of * box;
                const int here = min(boxes, (T - i * kP8Tokens + box - 1) / box);   // boxes that hold keys
                // Every lane waits for its own ring's stage.
                ok = __all_sync(0xffffffffu, wait(empty + 8 * s, ph));
                if (!ok) break;
                const bool skip = blockIdx.x == 0 && it == p.skip_tile && !is_v;    // injected fault: never loaded
                if ((lane & 7) == 0 && lane < 16 && !skip) mbar_arrive_expect_tx(full + 8 * s, here * box * D);
                __syncwarp();
                if (lane < 16 && box_of < here && !skip) {
                    // A page outside the pool is a slab out of range: zeros.
                    const int z = (unsigned)cur < (unsigned)p.num_pages ? cur * p.G + seg.g : -1;
                    tma_load_3d_hint(ring + s * TB + box_of * box * D, tm, full + 8 * s, 0, pos & (page_size - 1), z,
                                     pol);
                }
                __syncwarp();
                issued = it + 1;
                if (++s == S) s = 0, ph ^= 1;
            }
        }
        // Leave only once the last copies have landed.
        if (lane == 0 || lane == 8)
            for (int j = issued > S ? issued - S : 0; j < issued; ++j) {
                if (!is_v && blockIdx.x == 0 && j == p.skip_tile) continue;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full + 8 * (j % S), (j / S) & 1))
                    if (global_timer_ns() - t0 > tmo) break;
            }
        __syncwarp();
    } else if (warp == 9 || warp == 10) {
        // ----------------- products: S from one thread, O from another, so that
        // neither waits behind the other's operands
        if (lane == 0) {
            constexpr uint64_t kLayout = D == 128 ? 2 : 4;
            constexpr uint32_t kAtom = 8 * D;                               // 8 rows of K, V or Q
            bool ok = true, any = false;
            int s = 0, x = 0;
            uint32_t ph = 0, np[2] = {0, 0};
            if (warp == 9) {
                constexpr uint32_t kIdesc = p8_idesc(kP8Tokens, PS::kNs, false, false, false);
                const uint64_t k_desc = p8_desc(k_s, 16, kAtom, kLayout), q_desc = p8_desc(q_s, 16, kAtom, kLayout);
                int sg = 0;
                while (ok && walk.next(lens, seg)) {
                    ok = wait(q_full + 8 * (sg & 1), sg >> 1);
                    const uint64_t qd = q_desc + (sg & 1) * (PS::kQBytes >> 4);
                    for (int i = seg.i0; ok && i < seg.i1; ++i) {
                        // S_x of two tiles ago has been read.
                        ok = wait(s_free + 8 * x, (x ? np[1] : np[0]) + 1) && wait(k_full + 8 * s, ph);
                        if (!ok) break;
                        if (x) ++np[1]; else ++np[0];
                        tc_fence_after();
                        const uint64_t kd = k_desc + s * (TB >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            umma_f8(tmem + PS::kColS + x * PS::kNs, kd + kk * 2, qd + kk * 2, kIdesc, kk > 0 ? 1u : 0u);
                        umma_commit(s_full + 8 * x);
                        umma_commit(k_empty + 8 * s);
                        any = true;
                        x ^= 1;
                        if (++s == SK) s = 0, ph ^= 1;
                    }
                    if (ok) umma_commit(q_empty + 8 * (sg & 1));
                    ++sg;
                }
            } else {
                constexpr uint32_t kIdesc = p8_idesc(D, PS::kNp, true, true, true);
                const uint64_t v_desc = p8_desc(v_s, 16, kAtom, kLayout), p_desc = p8_desc(p_s, 128, 2048, 0);
                while (ok && walk.next(lens, seg)) {
                    bool first[2] = {true, true};
                    for (int i = seg.i0; i < seg.i1; ++i) {
                        ok = wait(v_full + 8 * s, ph) && wait(p_full + 8 * x, x ? np[1] : np[0]);
                        if (!ok) break;
                        const bool fresh = x ? first[1] : first[0];
                        if (x) ++np[1], first[1] = false; else ++np[0], first[0] = false;
                        tc_fence_after();
                        const uint64_t vd = v_desc + s * (TB >> 4), pd = p_desc + x * (PS::kPBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < kP8Tokens / 32; ++kk)
                            umma_f8(tmem + PS::kColO + x * PS::kNp, vd + kk * (2 * D), pd + kk * 32, kIdesc,
                                    (!fresh || kk > 0) ? 1u : 0u);
                        umma_commit(v_empty + 8 * s);
                        any = true;
                        x ^= 1;
                        if (++s == SV) s = 0, ph ^= 1;
                    }
                }
            }
            if (any) {
                const uint32_t bar = fin + 8 * (warp - 9);
                umma_commit(bar);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(bar, 0))
                    if (global_timer_ns() - t0 > tmo) {
                        atomicOr(p.status, kStatusTimeout);
                        break;
                    }
            }
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------ Q rows
        PagedFp8Split split = {-1, 0, 0, 0};
        long long at = plan->begin;
        int sg = 0;
        bool ok = true;
        while (ok && walk.next(lens, seg)) {
            if (seg.i0 == 0 && seg.i1 < seg.n)
                split = {seg.entry, seg.g, (int)(((at + seg.n) * plan->ctas - 1) / plan->total), 0};
            at += seg.i1 - seg.i0;
            const int buf = sg & 1;
            ok = warp_wait(q_empty + 8 * buf, ((sg >> 1) & 1) ^ 1, abort_flag, p.status, tmo);
            if (!ok) break;
            int b, rt;
            lens.split(seg.entry, b, rt);
            const int T = lens.tokens(b);
            const uint32_t qt = q_s + buf * PS::kQBytes;
            // Four lanes a row, eight rows at a time; the next rows are on
            // their way while these are split.
            constexpr int kVec = D / 32;          // 16-byte loads per lane: D / 4 elements
            const int part = lane & 3;
            uint4 next[kVec];
            int orow_next, tok_next;
            auto load_rows = [&](int r0) {
                tok_next = 0;
                orow_next = p8_out_row<RP>(p, b, rt, seg.g, r0 + (lane >> 2), &tok_next);
                const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)max(orow_next, 0) * D + part * (D / 4));
#pragma unroll
                for (int c = 0; c < kVec; ++c) next[c] = orow_next >= 0 ? src[c] : make_uint4(0, 0, 0, 0);
            };
            load_rows(0);
#pragma unroll 1
            for (int r0 = 0; r0 < RP; r0 += 8) {
                uint4 v[kVec];
#pragma unroll
                for (int c = 0; c < kVec; ++c) v[c] = next[c];
                const int orow = orow_next, tok = tok_next, r = r0 + (lane >> 2);
                if (r0 + 8 < RP) load_rows(r0 + 8);
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < kVec; ++c) {
                    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const bool bad = top >= 0x7f80u;              // an infinity or NaN: the whole row is NaN
                const int e = min(134 - max((int)(top >> 7), 1), 120);
                const float up = bad || top == 0 ? 0.f : pow2i(e);
#pragma unroll
                for (int c = 0; c < kVec; c += 2) {           // 16 elements: one 16-byte chunk of each row
                    const uint32_t w[8] = {v[c].x, v[c].y, v[c].z, v[c].w,
                                           v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float a = bad ? 0.f : __uint_as_float(w[k] << 16) * up;
                        const float d = bad ? 0.f : __uint_as_float(w[k] & 0xffff0000u) * up;
                        const uint32_t h = f32x2_to_e4m3x2(a, d);
                        const uint32_t hf = e4m3x2_to_f16x2((uint16_t)h);
                        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hf));
                        const uint32_t lw = f32x2_to_e4m3x2((a - back.x) * 16.f, (d - back.y) * 16.f);
                        if ((k & 1) == 0) hi[k / 2] = h, lo[k / 2] = lw;
                        else hi[k / 2] |= h << 16, lo[k / 2] |= lw << 16;
                    }
                    const uint32_t chunk = part * (D / 64) + c / 2;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t row = t * RP + r;
                        const uint32_t sw = D == 128 ? (row & 7) : ((row >> 1) & 3);
                        const uint32_t* x = t ? lo : hi;
                        st_shared_v4(qt + row * D + ((chunk ^ sw) << 4), make_uint4(x[0], x[1], x[2], x[3]));
                    }
                }
                if (part == 0) {
                    row_scale[buf * RP + r] = orow < 0 ? 0.f : bad ? __int_as_float(0x7fffffff)
                                                                 : p.scale_log2 * (top == 0 ? 1.f : pow2i(-e));
                    row_lim[buf * RP + r] = orow < 0 ? -1 : T - p.sq + tok;
                    row_out[buf * RP + r] = orow;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + 8 * buf);
            ++sg;
        }
        if (lane == 0) p.splits[blockIdx.x] = split;
        // Entries none of whose rows sees a key own no tile: out = 0, lse = -inf.
        for (int e = blockIdx.x; e < p.B * p.row_tiles; e += gridDim.x) {
            if (lens.tiles(e) > 0) continue;
            int b, rt;
            lens.split(e, b, rt);
            for (int x = 0; x < p.G * RP; ++x) {
                int tok;
                const int orow = p8_out_row<RP>(p, b, rt, x / RP, x % RP, &tok);
                if (orow < 0) continue;
                if (lane < D / 8) *reinterpret_cast<uint4*>(p.out + (size_t)orow * D + lane * 8) = make_uint4(0, 0, 0, 0);
                if (p.lse && lane == 0) p.lse[orow] = -INFINITY;
            }
        }
    } else {
        // ----------------------------------------- softmax groups, one thread a token
        const int x = warp >> 2, w4 = warp & 3;
        const int tok = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
        const uint32_t s_tm = lane_base + PS::kColS + x * PS::kNs;
        const uint32_t o_tm = lane_base + PS::kColO + x * PS::kNp;
        const uint32_t p_at = p_s + x * PS::kPBytes + tok * 16;
        float* const my_ref = neg_ref + x * RP;
        float2* const factor = factors + x * RP;
        int* const my_max = warp_max + x * 4 * (RP + 1);
        uint32_t n_tiles = 0, n_merge = 0;       // phases of s_full and p_full, of m_full
        int it0 = 0, sg = 0;                     // the CTA's tile number at the segment's start
        // The product of this group's tile `it` has completed.
        auto wait_product = [&](int it) { all_wait(v_empty + 8 * (it % SV), it / SV); };
        while (walk.next(lens, seg)) {
            int b, rt;
            lens.split(seg.entry, b, rt);
            const int T = lens.tokens(b);
            const int32_t* table = p.table + (size_t)b * p.max_pages;
            const float4* scale4 = reinterpret_cast<const float4*>(row_scale + (sg & 1) * RP);
            const int* lim = row_lim + (sg & 1) * RP;
            const int lim_min =                                             // every row sees keys up to here
                p.row_tiles == 1 ? T - p.sq : T - p.sq + (rt * RP) / p.heads_per_group;
            const int first_i = seg.i0 + ((it0 & 1) != x ? 1 : 0);          // this group's first tile
            auto page_of = [&](int i) {
                const int pos = i * kP8Tokens + tok;
                if (i >= seg.i1 || pos >= T) return -1;
                const int e = table[pos >> p.page_shift];
                return (unsigned)e < (unsigned)p.num_pages ? e : -1;
            };
            auto scales_of = [&](int page, int i, float& ks, float& vs) {
                ks = vs = 0.f;
                if (page >= 0) {
                    const int pos = i * kP8Tokens + tok;
                    const size_t at = ((size_t)page * p.G + seg.g) * p.blocks + ((pos & ((1 << p.page_shift) - 1)) >> 6);
                    ks = p.k_scale[at];
                    vs = p.v_scale[at];
                }
            };
            float ks, vs, l[RP];
            int ev = 0;
#pragma unroll
            for (int r = 0; r < RP; ++r) l[r] = 0.f;
            scales_of(page_of(first_i), first_i, ks, vs);
            int page_next = page_of(first_i + 2);
            bool first = true;
            // Also keeps a group without a tile here from running ahead.
            all_wait(q_full + 8 * (sg & 1), sg >> 1);
            for (int i = first_i; i < seg.i1; i += 2) {
                const int it = it0 + i - seg.i0;
                const int pos = i * kP8Tokens + tok;
                // The next tile's scales, and the page of the one after it.
                float ks_next, vs_next;
                scales_of(page_next, i + 2, ks_next, vs_next);
                page_next = page_of(i + 4);
                const bool edge = (i + 1) * kP8Tokens - 1 > lim_min;        // some row does not see all of it

                all_wait(s_full + 8 * x, n_tiles);
                tc_fence_after();
                float xs[RP];
                bool moves = first;
                {
                    uint32_t h[RP], lo[RP];
                    if constexpr (RP == 8) {
                        uint32_t t[16];
                        tmem_ld16(s_tm, t);
#pragma unroll
                        for (int r = 0; r < 8; ++r) h[r] = t[r], lo[r] = t[8 + r];
                    } else if constexpr (RP == 16) {
                        tmem_ld16(s_tm, h);
                        tmem_ld16(s_tm + 16, lo);
                    } else {
                        tmem_ld32(s_tm, h);
                        tmem_ld32(s_tm + 32, lo);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free + 8 * x);
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < RP; r += 4) {
                        const float4 f = scale4[r / 4];
                        const float4 m = *reinterpret_cast<const float4*>(my_ref + r);
                        const float fs[4] = {f.x, f.y, f.z, f.w}, ms[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            xs[r + k] = fmaf(__uint_as_float(lo[r + k]), 0.0625f, __uint_as_float(h[r + k])) * (fs[k] * ks);
                            if (edge && pos > lim[r + k]) xs[r + k] = -INFINITY;
                            top = fmaxf(top, xs[r + k] + ms[k]);
                        }
                    }
                    // A NaN or infinite scale makes its block's values NaN.
                    if (!(fabsf(vs) <= 3.402823466e38f)) vs = __int_as_float(0x7fffffff);
                    moves |= top > kP8Slack || fabsf(vs) * pow2i(-ev) > kP8ScaleSlack;
                }
                if (group_any(x, moves)) {
                    // Move the references: rows whose tile maximum is out of range.
                    int mine = 0;
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const int m = __reduce_max_sync(0xffffffffu, ordered(xs[r]));
                        if (lane == r) mine = m;
                    }
                    const uint32_t vb = __float_as_uint(fabsf(vs));
                    const uint32_t vtop = __reduce_max_sync(0xffffffffu, vb <= 0x7f7fffffu ? vb : 0u);
                    if (lane < RP) my_max[w4 * (RP + 1) + lane] = mine;
                    if (lane == 0) my_max[w4 * (RP + 1) + RP] = (int)vtop;
                    const float m_old = first || lane >= RP ? kP8Unseen : -my_ref[lane];
                    group_sync(x);
                    float m_new = m_old;
                    if (lane < RP) {
                        const float m = unordered(max(max(my_max[lane], my_max[RP + 1 + lane]),
                                                      max(my_max[2 * (RP + 1) + lane], my_max[3 * (RP + 1) + lane])));
                        if (m > m_old + kP8Slack) m_new = m;
                    }
                    const int vm = max(max(my_max[RP], my_max[2 * RP + 1]), max(my_max[3 * RP + 2], my_max[4 * RP + 3]));
                    // 2^-ev brings the largest scale to [0.5, 1).
                    const int ev_top = min(max((vm >> 23) - 126, -60), 126);
                    const int ev_new = first || __int_as_float(vm) * pow2i(-ev) > kP8ScaleSlack ? ev_top : ev;
                    const float alpha = fast_exp2(m_old - m_new);
                    const float alpha_o = first ? 0.f : alpha * pow2i(max(ev - ev_new, -126));
                    if (w4 == 0 && lane < RP) my_ref[lane] = -m_new;
                    ev = ev_new;
#pragma unroll
                    for (int r = 0; r < RP; ++r) l[r] *= __shfl_sync(0xffffffffu, alpha, r);
                    if (!first) {
                        wait_product(it - 2);     // and so every product of this group so far
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < PS::kNp / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o_tm + 16 * c, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) *
                                                       __shfl_sync(0xffffffffu, alpha_o, (16 * c + k) % RP));
                            tmem_st16(o_tm + 16 * c, o);
                        }
                        tmem_st_wait();
                    }
                    group_sync(x);
                }
                if (edge) {
                    // Rows of V past the length may hold anything: zero them. A
                    // NaN code in a key that only some rows see would reach the
                    // others as 0 * NaN: its row is zeroed too, and the rows that
                    // see it are made NaN through P.
                    const int s = it % SV;
                    all_wait(v_full + 8 * s, it / SV);
                    if (pos > lim_min) {
                        const uint32_t at = v_s + s * TB + tok * D;
                        bool clear = pos >= T;
                        if (!clear) {
                            uint32_t nan = 0;
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t u[4];
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                                             : "r"(at + 16 * c));
#pragma unroll
                                for (int k = 0; k < 4; ++k)   // a byte with its low seven bits set
                                    nan |= ((u[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                            }
                            clear = nan != 0;
                            if (clear) vs = __int_as_float(0x7fffffff);
                        }
                        if (clear)
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) st_shared_zero16(at + 16 * c);
                    }
                }
                const float vw = vs * pow2i(-ev) * kP8ProbScale;
                uint32_t packed[RP / 4][kP8Terms];       // a term of four rows
#pragma unroll
                for (int r = 0; r < RP; r += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(my_ref + r);
                    const float ms[4] = {m.x, m.y, m.z, m.w};
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float pr = fast_exp2(xs[r + k] + ms[k]);
                        l[r + k] += pr;
                        w[k] = pr * vw;
                        if (edge && pos > lim[r + k]) w[k] = 0.f;
                    }
                    uint32_t f0 = pack_f16x2(w[0], w[1]), f1 = pack_f16x2(w[2], w[3]);
#pragma unroll
                    for (int t = 0; t < kP8Terms; ++t) {
                        packed[r / 4][t] = __byte_perm(f0, f1, 0x7531);      // the four upper bytes
                        if (t + 1 < kP8Terms) {
                            f0 = e5m2_residual(f0);
                            f1 = e5m2_residual(f1);
                        }
                    }
                }
                // P's operand is free once the group's previous product is done.
                if (it >= 2) wait_product(it - 2);
                if (x == 1 && first) all_wait(m_empty, n_merge + 1);      // and handed-over O is read
                // Column term * RP + r; 16 columns of a token are 16 bytes.
#pragma unroll
                for (int c = 0; c < PS::kNp / 16; ++c) {
                    uint4 v;
                    if constexpr (RP == 8)
                        v = make_uint4(packed[0][2 * c], packed[1][2 * c], packed[0][2 * c + 1], packed[1][2 * c + 1]);
                    else {
                        constexpr int kHalf = RP / 16;
                        const int t = c / kHalf, q = (c % kHalf) * 4;
                        v = make_uint4(packed[q][t], packed[q + 1][t], packed[q + 2][t], packed[q + 3][t]);
                    }
                    st_shared_v4(p_at + c * 2048, v);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * x);
                ++n_tiles;
                first = false;
                ks = ks_next;
                vs = vs_next;
            }

            // ------------------------------------------------ end of a segment
            const int len = seg.i1 - seg.i0;
            const int cnt0 = (len + ((it0 & 1) == 0 ? 1 : 0)) / 2, cnt1 = len - cnt0;
            const bool both = cnt0 > 0 && cnt1 > 0;
            if ((x ? cnt1 : cnt0) > 0) {
                const float sum = reduce_rows<RP>(l, lane);
                if (lane < RP) reinterpret_cast<float*>(sums + x * RP + lane)[w4] = sum;
                group_sync(x);
                // This group's last tile is the segment's last or the one before.
                const int last = it0 + len - 1;
                wait_product((last & 1) == x ? last : last - 1);
                tc_fence_after();
                float o[RP];
#pragma unroll
                for (int r = 0; r < RP; ++r) o[r] = 0.f;
#pragma unroll
                for (int c = 0; c < PS::kNp / 16; ++c) {
                    uint32_t t[16];
                    tmem_ld16(o_tm + 16 * c, t);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[(16 * c + k) % RP] += __uint_as_float(t[k]);
                }
                tc_fence_before();
                // D = 64 products keep 16 of their rows in each warp's 32 lanes.
                const bool mine = D == 128 || lane < 16;
                const int dim = D == 128 ? tok : w4 * 16 + lane;
                const float unit = pow2i(ev) * (1.f / kP8ProbScale);
                if (both && x == 1) {
#pragma unroll
                    for (int r = 0; r < RP; ++r)
                        if (mine) stage_o[r * D + dim] = o[r] * unit;
                    if (tok < RP) {
                        const float4 q = sums[x * RP + tok];
                        other[tok] = make_float2(-my_ref[tok], q.x + q.y + q.z + q.w);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m_full);
                    ++n_merge;
                } else {
                    if (both) all_wait(m_full, n_merge);
                    const bool whole = seg.i0 == 0 && seg.i1 == seg.n;
                    float* slot = p.part + ((size_t)blockIdx.x * 2 + (seg.i0 == 0 ? 1 : 0)) * p8_slot_floats(RP, D);
                    const int* rows_out = row_out + (sg & 1) * RP;
                    if (tok < RP) {
                        const float4 q = sums[x * RP + tok];
                        float m = -my_ref[tok], ls = q.x + q.y + q.z + q.w, a0 = 1.f, a1 = 0.f;
                        if (both) {
                            const float2 u = other[tok];
                            const float top = fmaxf(m, u.x);
                            a0 = fast_exp2(m - top);
                            a1 = fast_exp2(u.x - top);
                            m = top;
                            ls = ls * a0 + u.y * a1;
                        }
                        if (whole) {
                            const bool some = ls > 0.f || ls != ls;
                            const float inv = some ? 1.f / ls : 0.f;
                            a0 *= inv;
                            a1 *= inv;
                            if (p.lse && rows_out[tok] >= 0)
                                p.lse[rows_out[tok]] = some ? (m + log2f(ls)) * 0.6931471805599453f : -INFINITY;
                        } else {
                            slot[RP * D + tok] = m;
                            slot[RP * D + RP + tok] = ls;
                        }
                        factor[tok] = make_float2(a0 * unit, a1);
                    }
                    group_sync(x);
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float2 f = factor[r];
                        float y = o[r] * f.x;
                        if (both && mine) y = fmaf(stage_o[r * D + dim], f.y, y);
                        if (!mine) continue;
                        if (!whole)
                            slot[r * D + dim] = y;
                        else if (rows_out[r] >= 0)
                            p.out[(size_t)rows_out[r] * D + dim] = (uint16_t)(pack_bf16x2(y, 0.f) & 0xffffu);
                    }
                    if (both) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(m_empty);
                        ++n_merge;
                    }
                }
                // The sums and references are read before the next segment writes them.
                group_sync(x);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty + 8 * (sg & 1));
            it0 += len;
            ++sg;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, PS::kTmemCols);
}

// Merges the partial results of the units that cross CTAs: one warp per row of
// the unit that CTA blockIdx.x began,
//     M = max m_c, L = sum l_c 2^(m_c - M), O = sum O_c 2^(m_c - M) / L.
template <int D, int RP>
__global__ void __launch_bounds__(128) gqa_paged_fp8_merge(const PagedFp8Params p) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const PagedFp8Split s = p.splits[blockIdx.x];
    if (s.entry < 0) return;
    const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int b = s.entry / p.row_tiles, rt = s.entry - b * p.row_tiles;
    int tok;
    const int orow = p8_out_row<RP>(p, b, rt, s.g, r, &tok);
    if (orow < 0) return;
    const int c0 = blockIdx.x, n = s.last_cta - c0 + 1;
    const size_t slot = p8_slot_floats(RP, D);
    // The first contributor's second slot, then every other's first.
    auto at = [&](int i) { return p.part + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * slot; };
    float top = kP8Unseen;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, at(i)[RP * D + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float l = 0.f;
    for (int i = lane; i < n; i += 32) l += at(i)[RP * D + RP + r] * fast_exp2(at(i)[RP * D + r] - top);
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    constexpr int kPer = D / 32;
    float y[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) y[k] = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float* src = at(i);
        const float a = fast_exp2(src[RP * D + r] - top);
        if constexpr (kPer == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + r * D + lane * 4);
            y[0] = fmaf(v.x, a, y[0]);
            y[1] = fmaf(v.y, a, y[1]);
            y[2] = fmaf(v.z, a, y[2]);
            y[3] = fmaf(v.w, a, y[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src + r * D + lane * 2);
            y[0] = fmaf(v.x, a, y[0]);
            y[1] = fmaf(v.y, a, y[1]);
        }
    }
    const bool some = l > 0.f || l != l;
    const float inv = some ? 1.f / l : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (size_t)orow * D + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) dst[k] = pack_bf16x2(some ? y[2 * k] * inv : 0.f, some ? y[2 * k + 1] * inv : 0.f);
    if (p.lse && lane == 0) p.lse[orow] = some ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int RP>
cudaError_t launch_paged_fp8(const PagedFp8Launch& a) {
    using PS = P8Shape<D, RP>;
    // The shared-memory opt-in is per function and per device.
    static std::atomic<unsigned long long> attr_set_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(attr_set_mask.load() & bit)) {
        e = cudaFuncSetAttribute(gqa_paged_fp8_kernel<D, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PS::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set_mask.fetch_or(bit);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(kP8Threads);
    cfg.dynamicSmemBytes = PS::kSmemBytes;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gqa_paged_fp8_kernel<D, RP>, a.tm_k, a.tm_v, a.p);
    if (e != cudaSuccess || a.grid == 1) return e;
    cfg.gridDim = dim3(a.grid, RP / 4);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, gqa_paged_fp8_merge<D, RP>, a.p);
}

template <int D>
cudaError_t launch_paged_fp8_rows(const PagedFp8Launch& a) {
    switch (p8_rows(a.p.R)) {
        case 8: return launch_paged_fp8<D, 8>(a);
        case 16: return launch_paged_fp8<D, 16>(a);
        default: return launch_paged_fp8<D, 32>(a);
    }
}

}  // namespace gqa
