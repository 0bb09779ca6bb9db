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
//   w = fp16(p * v_scale * 2^c) = t0 + t1 / 8 + t2 / 64 + t3 / 512, e5m2: a term
//     is the upper byte of the fp16 residual (its first 3 significant bits), the
//     next residual the exact difference times 8, which fits fp16 again. The 4
//     terms are all of w, subnormals too: w is p * v_scale within half an fp16
//     step, 2^-11 of itself or 2^-25, where w is 1024..2048 for p = 1 and the
//     largest scale. (Without the factors what lies below e5m2's least step,
//     2^-16, was dropped: 2^17 keys with a hundredth of the weight behind a key
//     with the rest came out 3 % low, 2^20 of them 22 %.) No conversion
//     instruction is needed; an e4m3 split takes two per term and pair, and
//     those, at a quarter of the rate, took half of a tile's time.
// The extra columns cost nothing: up to N = 128 a product of M = 128 takes the
// 64 cycles that reading its K or V rows takes.
//
// Softmax, one thread per token: x = s * scale2 * k_scale (base 2), p = 2^(x - m)
// with a reference m per row that moves only when a score exceeds it by more
// than 4 (then O is rescaled in tensor memory), so that tiles need no maximum
// across threads: one vote. The sum l is kept per thread until the end. v_scale
// enters p through a power of two 2^c that follows the largest scale seen.
//
// Work: the tiles of all units, end to end, are shared equally by the CTAs (one
// per SM; units of unlike lengths count a few tiles more for their end). A unit
// that crosses CTAs leaves (O, m, l) per CTA in the workspace; the CTA that
// arrives last merges them. Per CTA: two groups of four softmax warps (with 32
// rows two such pairs, 16 rows each) take alternate tiles. One warp brings K,
// another V (a TMA box per page, in the swizzle of the operand layout; one warp
// issues a box in 65 cycles, two warps two); the latter also fetches the blocks'
// scales, ahead of V by a chunk of tiles (behind a saturated HBM a lookup of page
// and scale takes longer than a tile). Two warps issue the products. Every wait
// is bounded, as in the other kernels.
//
// What bounds it. Bytes: the cache, once. A tile of 8 rows takes 0.3 us, one of 32
// rows 0.70 to 0.75 us (a softmax warp's chain of load, vote, exponentials and
// four terms is 2500 cycles, two groups at a time), against 0.62 to 0.74 us for
// a tile's 32 KB from HBM shared by 128 to 152 SMs. Around the tiles: 2 us of
// launch, 1.5 us of plan, 2 us until the first softmax, and where a unit is
// split 4 to 6 us for its parts (stores, one atomic, the last arriver's merge).
// Every 32 rows walk their keys again, so chunks of a prompt are bound by the
// softmax chain: a quarter of the bf16 rate from 512 new tokens on.
// Measured on one GB300 (HBM copy 6.77 TB/s, SM clock 2070 MHz), B x H/G heads,
// tokens, page; rates by the lengths that were read:
//   16 x 32/8, D 128, 4096, 64           25.4 us, 5.3 TB/s (6.5 TB/s at 16384 tokens)
//   64 x 32/1, D 128, 8192, 32           33.8 us, 4.0 TB/s
//   1 x 64/8, D 128, 131072, 16          52.6 us, 5.1 TB/s
//   64 x 64/8, 4 new tokens, D 128, 512 to 32768, 64   322 us, 6.5 TB/s (8 rows 6.9)
//   64 x 64/8, 4 new tokens, D 128, up to 4096, 64     79.5 us, 3.15 TB/s (16 rows
//                                        70 us, 8 rows 52 us)
//   16 x 32/8, D 64, 16384, 64           75 us, 3.6 TB/s
//   1 x 32/8, 64 new tokens, D 64, 4096, 64            23.7 us (4.7 MB: latency)
//   4 x 32/8, 2048 new tokens, D 128, 8192, 64         2290 us, 420 TFLOP/s (the
//                                        bf16 prefill kernel 851 us)
// With 32 rows and D 128 the registers are one short: 8 bytes spilled, 20 read.
// Tried and slower: asking for a barrier's phase ahead of its wait (MQA end +0.3
// us), running the merge once without effect to fetch its instructions (+0.7 us),
// 152 CTAs with uneven shares where 128 share equal units evenly (+2.8 us), the
// next unit's queries split between this one's tiles (ragged +12 to +35 us: any
// longer loader loop slows every tile), a stage more in each ring (no change).
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "gqa_device.cuh"
#include "gqa_paged_fp8.h"
#include "gqa_paged_plan.cuh"
#include "tcgen05.cuh"

namespace gqa {

constexpr int kP8ScaleChunk = 4;          // tiles whose scales are fetched together,
constexpr int kP8ScaleChunks = 8;         // and how many such chunks a CTA keeps
constexpr int kP8Terms = 4;               // e5m2 columns per probability
constexpr float kP8Slack = 4.0f;          // p <= 2^4 before the reference moves
constexpr float kP8ProbScale = 2048.0f;   // p * v_scale * 2^-ev * 2048 <= 16 * 1.75 * 2048 = 57344
constexpr float kP8ScaleSlack = 1.75f;
constexpr float kP8Unseen = -3.402823466e38f;   // reference of a row that has seen no key

template <int D, int RP>
struct P8Shape {
    static constexpr int kTileBytes = kP8Tokens * D;              // K or V of one tile
    static constexpr int kParts = RP == 32 ? 2 : 1;               // row parts, each with its own warps
    static constexpr int kRows = RP / kParts;                     // rows per softmax thread
    static constexpr int kSoftWarps = 8 * kParts;
    static constexpr int kThreads = (kSoftWarps + 4) * 32;
    static constexpr int kNs = 2 * RP;                            // columns of S: hi, lo
    static constexpr int kNp = kP8Terms * RP;                     // columns of O
    static constexpr int kQBytes = kNs * D;
    static constexpr int kPBytes = kP8Tokens * kNp;
    // The rings take what the rest leaves of 227 KB. A V tile is held from its
    // copy to P V, a K tile only to S, so V gets more stages.
    static constexpr int kStagesK = (D == 128 ? 1 : 2) * (RP == 32 ? 4 : 5);
    static constexpr int kStagesV = (D == 128 ? 1 : 2) * (RP == 32 ? 5 : 7);
    static constexpr int kBars = 2 * (kStagesK + kStagesV) + 16 + kP8ScaleChunks;
    static constexpr int kRowInfoBytes = 2 * 3 * RP * 4;
    static constexpr int kRefBytes = 2 * RP * 4;
    static constexpr int kWarpMaxBytes = 2 * kParts * 4 * (kRows + 1) * 4;
    static constexpr int kSumBytes = 2 * RP * 16;
    static constexpr int kMergeBytes = 3 * RP * 8;                // (m, l) handed over; each group's row factors
    static constexpr int kLenBytes = kP8LenCopy * 4 + 16;         // and the plan's padding
    static constexpr int kScaleBytes = kP8ScaleChunks * kP8ScaleChunk * 16 * 4;
    static constexpr int kMiscBytes = 320;
    static constexpr int kSmemBytes = 1024 + (kStagesK + kStagesV) * kTileBytes + 2 * kQBytes + 2 * kPBytes +
                                      kRowInfoBytes + kRefBytes + kWarpMaxBytes + kSumBytes + kMergeBytes +
                                      kLenBytes + kScaleBytes + kMiscBytes + 8 * kBars;
    // A group hands its O over in its own P operand, which its last product has read.
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

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
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

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}

// Two runs of 16 columns, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
          "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
          "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
        : "r"(ta), "r"(tb)
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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

template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_ld8(taddr, r); else tmem_ld16(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_st8(taddr, r); else tmem_st16(taddr, r);
}

// ------------------------------------------------------------ e4m3 and fp16

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 times what is left of two fp16 values without their first e5m2 terms: exact,
// and at most 8 * (2^-2 - 2^-10) of the value's power of two, so in range.
constexpr float kP8TermStep = 8.0f;
__device__ __forceinline__ uint32_t e5m2_residual(uint32_t f) {
    const uint32_t t = f & 0xff00ff00u;
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&f), *reinterpret_cast<const __half2*>(&t));
    const __half2 r = __hmul2(d, __float2half2_rn(kP8TermStep));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Floats to integers of the same order, and back.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // |e| <= 126

// Two fp32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma_x2(float2 a, float2 b, float2 c) {
    unsigned long long x, y, z, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
    return a;
}
__device__ __forceinline__ float2 mul_x2(float2 a, float2 b) {
    unsigned long long x, y, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
    return a;
}
__device__ __forceinline__ float2 add_x2(float2 a, float2 b) {
    unsigned long long x, y, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
    return a;
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
    const int s = p.by_heads(rr);
    *s_tok = s;
    return (b * p.sq + s) * p.H + g * p.heads_per_group + (rr - s * p.heads_per_group);
}

// One group's merge of rows [r0, r0 + RH) of a unit that n CTAs from c0 on hold
// parts of; the first CTA's part is in its second slot, every other's in its
// first. A thread merges four columns of some rows, several parts at a time, all
// of their loads under way at once.
template <int D, int RP, int RH>
__device__ __noinline__ void p8_merge(const PagedFp8Params& p, int c0, int n, int r0, int tok, const int* rows_out) {
    constexpr int kItems = RH * D / 4 / 128;      // 1 to 4
    constexpr int kAtOnce = kItems > 2 ? 2 : 4;
    const size_t slot = p8_slot_floats(RP, D);
    auto at = [&](int i) { return p.part + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * slot; };
    float top[kItems], l[kItems], y[kItems][4];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        top[j] = kP8Unseen;
        l[j] = y[j][0] = y[j][1] = y[j][2] = y[j][3] = 0.f;
    }
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
        float m[kItems][kAtOnce], s[kItems][kAtOnce];
        float4 v[kItems][kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                const int item = j * 128 + tok, r = r0 + item / (D / 4), d = item % (D / 4) * 4;
                m[j][k] = kP8Unseen;
                s[j][k] = 0.f;
                v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + k < n) {
                    const float* part = at(i0 + k);
                    m[j][k] = __ldcg(part + RP * D + r);
                    s[j][k] = __ldcg(part + RP * D + RP + r);
                    v[j][k] = __ldcg(reinterpret_cast<const float4*>(part + r * D + d));
                }
            }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            float t = top[j];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) t = fmaxf(t, m[j][k]);
            const float a = fast_exp2(top[j] - t);
            top[j] = t;
            l[j] *= a;
#pragma unroll
            for (int c = 0; c < 4; ++c) y[j][c] *= a;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (i0 + k >= n) continue;
                const float w = fast_exp2(m[j][k] - t);
                l[j] = fmaf(s[j][k], w, l[j]);
                y[j][0] = fmaf(v[j][k].x, w, y[j][0]);
                y[j][1] = fmaf(v[j][k].y, w, y[j][1]);
                y[j][2] = fmaf(v[j][k].z, w, y[j][2]);
                y[j][3] = fmaf(v[j][k].w, w, y[j][3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int item = j * 128 + tok, d = item % (D / 4) * 4, orow = rows_out[item / (D / 4)];
        if (orow < 0) continue;
        const bool some = l[j] > 0.f || l[j] != l[j];
        const float inv = __fdividef(1.f, l[j]);
        uint2 o = make_uint2(0, 0);
        if (some) {
            o.x = pack_bf16x2(y[j][0] * inv, y[j][1] * inv);
            o.y = pack_bf16x2(y[j][2] * inv, y[j][3] * inv);
        }
        *reinterpret_cast<uint2*>(p.out + (size_t)orow * D + d) = o;
        if (p.lse && d == 0) p.lse[orow] = some ? (top[j] + __log2f(l[j])) * 0.6931471805599453f : -INFINITY;
    }
}

// ------------------------------------------------------------------- kernel

// The threads of a group meet (and agree whether any of them votes), on the
// CTA's named barriers. No softmax thread leaves its loop early, whatever a
// bounded wait reported, so all of a group's warps always arrive.
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ unsigned long long add_acq_rel(unsigned long long* at, unsigned long long v) {
    unsigned long long old;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(old) : "l"(at), "l"(v) : "memory");
    return old;
}
__device__ __forceinline__ unsigned long long cas_acq_rel(unsigned long long* at, unsigned long long seen,
                                                          unsigned long long v) {
    unsigned long long was;
    asm volatile("atom.cas.acq_rel.gpu.global.b64 %0, [%1], %2, %3;" : "=l"(was) : "l"(at), "l"(seen), "l"(v) : "memory");
    return was;
}

// Counts one arrival on a counter that holds (tag << 16 | count); one with
// another tag counts from zero. True for the last of n, which leaves a count
// of zero: a captured call is replayed with its tag.
__device__ __forceinline__ bool arrive_last(unsigned long long* counter, unsigned long long tag, unsigned n) {
    const unsigned long long zero = tag << 16;
    unsigned count;
    const unsigned long long old = add_acq_rel(counter, 1ull);
    if (old >> 16 == tag) {
        count = (unsigned)(old & 0xffffu) + 1;
    } else {
        unsigned long long seen = *reinterpret_cast<volatile unsigned long long*>(counter);
        while (true) {
            if (seen >> 16 == tag) {           // another arrival has tagged it: its count lacks this one
                count = (unsigned)(add_acq_rel(counter, 1ull) & 0xffffu) + 1;
                break;
            }
            const unsigned long long was = cas_acq_rel(counter, seen, zero | 1ull);
            if (was == seen) {
                count = 1;
                break;
            }
            seen = was;
        }
    }
    if (count != n) return false;
    atomicExch(counter, zero);
    return true;
}

// Gives a counter the call's tag ahead of its arrivals, which then take one
// atomic each instead of three. No arrival is lost: one whose add this
// overwrites finds the tag and adds again.
__device__ __forceinline__ void tag_counter(unsigned long long* counter, unsigned long long tag) {
    const unsigned long long seen = *reinterpret_cast<volatile unsigned long long*>(counter);
    if (seen >> 16 != tag) atomicCAS(counter, seen, tag << 16);
}

template <int D, int RP>
__global__ void __launch_bounds__(P8Shape<D, RP>::kThreads, 1)
    gqa_paged_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PagedFp8Params p) {
    using PS = P8Shape<D, RP>;
    constexpr int SK = PS::kStagesK, SV = PS::kStagesV, RH = PS::kRows, SW = PS::kSoftWarps;
    constexpr uint32_t TB = PS::kTileBytes;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t k_s = base, v_s = k_s + SK * TB, q_s = v_s + SV * TB, p_s = q_s + 2 * PS::kQBytes;
    unsigned char* gen = smem_raw + (p_s + 2 * PS::kPBytes - raw);
    float* const handed = reinterpret_cast<float*>(gen - 2 * PS::kPBytes);   // O of each group, in its P
    // Rows of the unit in q buffer i: scale2 * 2^-e, last visible key, output row.
    float* row_scale = reinterpret_cast<float*>(gen);                     // [2][RP]
    int* row_lim = reinterpret_cast<int*>(row_scale + 2 * RP);            // [2][RP]
    int* row_out = row_lim + 2 * RP;                                      // [2][RP]
    gen += PS::kRowInfoBytes;
    float4* sums = reinterpret_cast<float4*>(gen);                        // [2][RP], one component a warp
    gen += PS::kSumBytes;
    float* neg_ref = reinterpret_cast<float*>(gen);                       // [2][RP]: -m
    gen += PS::kRefBytes;
    float2* other = reinterpret_cast<float2*>(gen);                       // [RP]: (m, l) handed over
    float2* factors = other + RP;                                         // [2][RP]: weights of the groups' O
    gen += PS::kMergeBytes;
    float* scale_ring = reinterpret_cast<float*>(gen);                    // [slots][8 of K, 8 of V]
    gen += PS::kScaleBytes;
    int* warp_max = reinterpret_cast<int*>(gen);                          // [2][parts][4][RH + 1]
    gen += PS::kWarpMaxBytes;
    int* len_copy = reinterpret_cast<int*>(gen);
    gen += PS::kLenBytes;
    P8Plan* plan_s = reinterpret_cast<P8Plan*>(gen);                      // 48 bytes
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + 64);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gen + 68);
    volatile int* last_flag = reinterpret_cast<volatile int*>(gen + 72);  // [4]
    long long* warp_sum = reinterpret_cast<long long*>(gen + 96);         // [20]
    gen += PS::kMiscBytes;
    const uint32_t bar0 = smem_addr(gen);
    const uint32_t k_full = bar0, k_empty = k_full + 8 * SK, v_full = k_empty + 8 * SK, v_empty = v_full + 8 * SV;
    const uint32_t q_full = v_empty + 8 * SV, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, s_free = s_full + 16, p_full = s_free + 16;
    const uint32_t m_full = p_full + 16, m_empty = m_full + 16, fin = m_empty + 16;
    const uint32_t sc_full = fin + 16;

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
            mbar_init(q_full + 8 * x, RP / 8);          // eight rows a time
            mbar_init(q_empty + 8 * x, SW + 1);         // the softmax warps and the products
            mbar_init(s_full + 8 * x, 1);
            mbar_init(s_free + 8 * x, 4 * PS::kParts);
            mbar_init(p_full + 8 * x, 4 * PS::kParts);
            mbar_init(fin + 8 * x, 1);
            mbar_init(m_full + 8 * x, 4);
            mbar_init(m_empty + 8 * x, 4);
        }
        for (int c = 0; c < kP8ScaleChunks; ++c) mbar_init(sc_full + 8 * c, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    // No output row yet: after an expired wait a segment may end whose rows were
    // never split, and writes nothing then.
    if (threadIdx.x < 2 * RP) row_out[threadIdx.x] = -1;
    if (warp == SW + 1) {
        tmem_alloc(smem_addr(tmem_slot), PS::kTmemCols);
        tmem_relinquish();
    }
    if (warp == SW && lane < 2) tma_prefetch_desc(lane ? &tm_v : &tm_k);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait_primary();
    P8Walk<RP> walk;
    if (p.small_plan) {
        if (threadIdx.x < 128) len_copy[threadIdx.x] = (int)threadIdx.x < p.B ? lens.global(threadIdx.x) : 0;
        if (threadIdx.x == 0) len_copy[kP8LenCopy + 1] = 0;
        __syncthreads();
        const P8Plan plan = p8_small_plan<RP>(lens);
        // Kept in shared memory (every warp writes the same) rather than in
        // registers until a split unit's end needs it.
        if (lane == 0) *plan_s = plan;
        __syncwarp();
        walk = {plan.left, plan.entry, plan.g, plan.off};
    } else {
        p8_make_plan<RP, PS::kThreads>(p, len_copy, plan_s, warp_sum);
        __syncthreads();
        walk = {plan_s->left, plan_s->entry, plan_s->g, plan_s->off};
    }
    P8Segment seg;
    // Bounded waits of one thread, and of a softmax warp: all its lanes poll,
    // and all go on when the limit runs out.
    auto wait = [&](uint32_t bar, uint32_t n) { return wait_phase(bar, n & 1, abort_flag, p.status, tmo); };
    auto all_wait = [&](uint32_t bar, uint32_t n) {
        if (!mbar_try_wait(bar, n & 1) && !*abort_flag) wait_phase(bar, n & 1, abort_flag, p.status, tmo);
        __syncwarp();
    };

    // One ring's copies of a segment's tiles, a lane per page; every lane of the
    // calling warp takes part. `between` runs before each tile.
    const int page_size = 1 << p.page_shift;
    auto load_tiles = [&](const P8Segment& seg, int b, int T, const CUtensorMap* tm, uint32_t ring, int S, uint32_t full,
                          uint32_t empty, int skip_tile, uint64_t pol, int& it, int& s, uint32_t& ph, auto between) {
        const int box = min(page_size, kP8Tokens);              // rows of a copy
        const int boxes = kP8Tokens / box;
        const int32_t* row = p.table + (size_t)b * p.max_pages;
        // The table is read 32 entries at a time, a lane each, and the next 32
        // are on their way.
        int first = (seg.i0 * kP8Tokens) >> p.page_shift;
        const int last = (min(T, seg.i1 * kP8Tokens) - 1) >> p.page_shift;
        auto entries = [&](int e) { return e + lane <= last ? row[e + lane] : -1; };
        int cur = entries(first), nxt = entries(first + 32);
        for (int i = seg.i0; i < seg.i1; ++i, ++it) {
            if (((i * kP8Tokens) >> p.page_shift) - first >= 32) {
                first += 32;
                cur = nxt;
                nxt = entries(first + 32);
            }
            between(i);
            const int pos = i * kP8Tokens + lane * box;
            const int page = __shfl_sync(0xffffffffu, cur, ((pos >> p.page_shift) - first) & 31);
            const int here = min(boxes, (T - i * kP8Tokens + box - 1) / box);   // boxes that hold keys
            if (!warp_wait(empty + 8 * s, ph, abort_flag, p.status, tmo)) return false;
            if (it != skip_tile) {
                if (lane == 0) mbar_arrive_expect_tx(full + 8 * s, here * box * D);
                __syncwarp();
                if (lane < here)
                    // A page outside the pool is a slab out of range: zeros.
                    tma_load_3d_hint(ring + s * TB + lane * box * D, tm, full + 8 * s, 0, pos & (page_size - 1),
                                     (unsigned)page < (unsigned)p.num_pages ? page * p.G + seg.g : -1, pol);
            }
            __syncwarp();
            if (++s == S) s = 0, ph ^= 1;
        }
        return true;
    };
    // A loader leaves only once its last copies have landed.
    auto drain = [&](uint32_t full, int S, int issued, int skip_tile) {
        if (lane == 0)
            for (int j = issued > S ? issued - S : 0; j < issued; ++j) {
                if (j == skip_tile) continue;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(full + 8 * (j % S), (j / S) & 1))
                    if (global_timer_ns() - t0 > tmo) break;
            }
        __syncwarp();
    };

    // Eight query rows of a unit at a time, by one warp, four lanes a row: their
    // loads, and their split into q buffer `buf`, which arrives on its barrier.
    constexpr int kVec = D / 32;                  // 16-byte loads per lane: D / 4 elements
    struct QRows {
        uint4 v[kVec];
        int orow, tok;
    };
    auto load_rows = [&](int b, int rt, int g, int r0) {
        QRows q;
        q.tok = 0;
        q.orow = p8_out_row<RP>(p, b, rt, g, r0 + (lane >> 2), &q.tok);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (size_t)max(q.orow, 0) * D + (lane & 3) * (D / 4));
#pragma unroll
        for (int c = 0; c < kVec; ++c) q.v[c] = q.orow >= 0 ? src[c] : make_uint4(0, 0, 0, 0);
        return q;
    };
    auto split_rows = [&](const QRows& q, int T, int buf, int r0) {
        const uint32_t qt = q_s + buf * PS::kQBytes;
        const int part = lane & 3, r = r0 + (lane >> 2), orow = q.orow, tok = q.tok;
        const uint4 (&v)[kVec] = q.v;
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool bad = top >= 0x7f80u;          // an infinity or NaN: the whole row is NaN
        const int e = min(134 - max((int)(top >> 7), 1), 120);
        const float up = bad || top == 0 ? 0.f : pow2i(e);
#pragma unroll
        for (int c = 0; c < kVec; c += 2) {       // 16 elements: one 16-byte chunk of each row
            const uint32_t w[8] = {v[c].x, v[c].y, v[c].z, v[c].w, v[c + 1].x, v[c + 1].y, v[c + 1].z, v[c + 1].w};
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
            row_scale[buf * RP + r] =
                orow < 0 ? 0.f : bad ? __int_as_float(0x7fffffff) : p.scale_log2 * (top == 0 ? 1.f : pow2i(-e));
            row_lim[buf * RP + r] = orow < 0 ? -1 : T - p.sq + tok;
            row_out[buf * RP + r] = orow;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * buf);
    };

    // The first segment's rows are split by softmax warps, which have nothing
    // else to do yet, eight rows each; those of later segments by the K loader,
    // which is ahead of the products, in turn, 1300 cycles per eight rows. With
    // 32 rows that is too long for short segments: the softmax group that is
    // done first with a segment takes them. 512 units of 1 to 4096 tokens, 32
    // rows: loader 82, group 77 us; 8 rows: 58 and 66 us.
    constexpr bool kLoaderSplits = RP < 32;
    if (warp < RP / 8) {
        P8Walk<RP> peek = walk;
        if (peek.next(lens, seg)) {
            int b, rt;
            lens.split(seg.entry, b, rt);
            split_rows(load_rows(b, rt, seg.g, warp * 8), lens.tokens(b), 0, warp * 8);
        }
    }

    if (warp == SW) {
        // ------------------------------------------------ K loader, Q rows
        const int skip_tile = blockIdx.x == 0 ? p.skip_tile : -1;      // injected fault: never loaded
        const uint64_t pol = l2_policy_evict_first();
        int it = 0, s = 0, sg = 0;
        uint32_t ph = 1;
        bool ok = true;
        while (ok && walk.next(lens, seg)) {
            int b, rt;
            lens.split(seg.entry, b, rt);
            if (kLoaderSplits && sg > 0) {
                QRows next = load_rows(b, rt, seg.g, 0);
                ok = warp_wait(q_empty + 8 * (sg & 1), ((sg >> 1) & 1) ^ 1, abort_flag, p.status, tmo);
                if (!ok) break;
#pragma unroll 1
                for (int r0 = 0; r0 < RP; r0 += 8) {
                    const QRows q = next;
                    if (r0 + 8 < RP) next = load_rows(b, rt, seg.g, r0 + 8);
                    split_rows(q, lens.tokens(b), sg & 1, r0);
                }
            }
            ++sg;
            ok = load_tiles(seg, b, lens.tokens(b), &tm_k, k_s, SK, k_full, k_empty, skip_tile, pol, it, s, ph,
                            [](int) {});
        }
        drain(k_full, SK, it, skip_tile);
    } else if (warp == SW + 1 || warp == SW + 2) {
        // ----------------- products: S from one warp, O from another, so that
        // neither waits behind the other's operands. The warp waits as a whole
        // and one thread issues; what the instructions take is made uniform.
        constexpr uint64_t kLayout = D == 128 ? 2 : 4;
        constexpr uint32_t kAtom = 8 * D;                               // 8 rows of K, V or Q
        bool ok = true, any = false;
        int s = 0, x = 0;
        uint32_t ph = 0, np[2] = {0, 0};
        const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
        auto wait_warp = [&](uint32_t bar, uint32_t n) {
            return __all_sync(0xffffffffu, wait(bar, n)) != 0;
        };
        if (warp == SW + 1) {
            constexpr uint32_t kIdesc = p8_idesc(kP8Tokens, PS::kNs, false, false, false);
            const uint64_t k_desc = p8_desc(k_s, 16, kAtom, kLayout), q_desc = p8_desc(q_s, 16, kAtom, kLayout);
            int sg = 0, chunk = 0;
            while (ok && walk.next(lens, seg)) {
                ok = wait_warp(q_full + 8 * (sg & 1), sg >> 1);
                for (int i = seg.i0; ok && i < seg.i1; ++i) {
                    // The scales of this tile and the next three are there, and
                    // S_x of two tiles ago has been read.
                    if ((i - seg.i0) % kP8ScaleChunk == 0) {
                        ok = wait_warp(sc_full + 8 * (chunk % kP8ScaleChunks), chunk / kP8ScaleChunks);
                        ++chunk;
                    }
                    ok = ok && wait_warp(s_free + 8 * x, (x ? np[1] : np[0]) + 1) && wait_warp(k_full + 8 * s, ph);
                    if (!ok) break;
                    if (x) ++np[1]; else ++np[0];
                    tc_fence_after();
                    const int su = __shfl_sync(0xffffffffu, s, 0), xu = __shfl_sync(0xffffffffu, x, 0);
                    const int bu = __shfl_sync(0xffffffffu, sg & 1, 0);
                    if (elect_one()) {
                        const uint64_t kd = k_desc + su * (TB >> 4), qd = q_desc + bu * (PS::kQBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 32; ++kk)
                            umma_f8(tmem_u + PS::kColS + xu * PS::kNs, kd + kk * 2, qd + kk * 2, kIdesc, kk > 0 ? 1u : 0u);
                        umma_commit(s_full + 8 * xu);
                        umma_commit(k_empty + 8 * su);
                        if (i + 1 == seg.i1) umma_commit(q_empty + 8 * bu);
                    }
                    __syncwarp();
                    any = true;
                    x ^= 1;
                    if (++s == SK) s = 0, ph ^= 1;
                }
                ++sg;
            }
        } else {
            // This warp has nothing to do until the first P: the counters of the
            // unit that this CTA may start.
            if (lane < PS::kParts) tag_counter(p.counters + (size_t)blockIdx.x * PS::kParts + lane, p.tag);
            __syncwarp();
            constexpr uint32_t kIdesc = p8_idesc(D, PS::kNp, true, true, true);
            const uint64_t v_desc = p8_desc(v_s, 16, kAtom, kLayout), p_desc = p8_desc(p_s, 128, 2048, 0);
            while (ok && walk.next(lens, seg)) {
                bool first[2] = {true, true};
                for (int i = seg.i0; i < seg.i1; ++i) {
                    ok = wait_warp(v_full + 8 * s, ph) && wait_warp(p_full + 8 * x, x ? np[1] : np[0]);
                    if (!ok) break;
                    const bool fresh = x ? first[1] : first[0];
                    if (x) ++np[1], first[1] = false; else ++np[0], first[0] = false;
                    tc_fence_after();
                    const int su = __shfl_sync(0xffffffffu, s, 0), xu = __shfl_sync(0xffffffffu, x, 0);
                    const int fu = __shfl_sync(0xffffffffu, fresh ? 1 : 0, 0);
                    if (elect_one()) {
                        const uint64_t vd = v_desc + su * (TB >> 4), pd = p_desc + xu * (PS::kPBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < kP8Tokens / 32; ++kk)
                            umma_f8(tmem_u + PS::kColO + xu * PS::kNp, vd + kk * (2 * D), pd + kk * 32, kIdesc,
                                    (fu == 0 || kk > 0) ? 1u : 0u);
                        umma_commit(v_empty + 8 * su);
                    }
                    __syncwarp();
                    any = true;
                    x ^= 1;
                    if (++s == SV) s = 0, ph ^= 1;
                }
            }
        }
        // elect_one picks the same thread each time: its commit covers all of the warp's products.
        if (any && elect_one()) {
            const uint32_t bar = fin + 8 * (warp - SW - 1);
            umma_commit(bar);
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar, 0))
                if (global_timer_ns() - t0 > tmo) {
                    atomicOr(p.status, kStatusTimeout);
                    break;
                }
        }
        __syncwarp();
    } else if (warp == SW + 3) {
        // --------------------------------------------------- scales, V loader
        const int block = min(page_size, 64);     // tokens of a scale
        const uint64_t pol = l2_policy_evict_first();
        int sg = 0, chunk = 0, it = 0, s = 0;
        uint32_t ph = 1;
        bool ok = true;
        while (ok && walk.next(lens, seg)) {
            const int buf = sg & 1;
            int b, rt;
            lens.split(seg.entry, b, rt);
            const int T = lens.tokens(b);
            // Scales of the segment's tiles, a chunk of four at a time: lane
            // (tile, block); pages two chunks ahead, scales one.
            const int32_t* table = p.table + (size_t)b * p.max_pages;
            auto pos_of = [&](int i) {           // this lane's position in the chunk at tile i, -1: none
                i += lane >> 3;
                const int pos = i * kP8Tokens + (lane & 7) * block;
                return i < seg.i1 && (lane & 7) * block < kP8Tokens && pos < T ? pos : -1;
            };
            auto page_of = [&](int pos) {
                const int e = pos >= 0 ? table[pos >> p.page_shift] : -1;
                return (unsigned)e < (unsigned)p.num_pages ? e : -1;
            };
            float ks, vs;
            auto fetch_scales = [&](int pos, int page) {
                ks = vs = 0.f;
                if (page >= 0) {
                    const size_t at = ((size_t)page * p.G + seg.g) * p.blocks + ((pos & (page_size - 1)) >> 6);
                    ks = __ldg(p.k_scale + at);
                    vs = __ldg(p.v_scale + at);
                }
            };
            auto store_scales = [&]() {
                float* to = scale_ring + ((chunk % kP8ScaleChunks) * kP8ScaleChunk + (lane >> 3)) * 16 + (lane & 7);
                to[0] = ks;
                to[8] = vs;
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full + 8 * (chunk % kP8ScaleChunks));
                ++chunk;
            };
            const int page_first = page_of(pos_of(seg.i0));
            ok = warp_wait(q_empty + 8 * buf, ((sg >> 1) & 1) ^ 1, abort_flag, p.status, tmo);
            if (!ok) break;
            fetch_scales(pos_of(seg.i0), page_first);
            int page_next = page_of(pos_of(seg.i0 + kP8ScaleChunk));
            ++sg;
            // Slots are reused eight chunks later: by then this warp, which is
            // at most two segments and kStagesV tiles ahead of the products,
            // has seen the tiles done whose scales they held.
            store_scales();
            fetch_scales(pos_of(seg.i0 + kP8ScaleChunk), page_next);
            page_next = page_of(pos_of(seg.i0 + 2 * kP8ScaleChunk));
            ok = load_tiles(seg, b, T, &tm_v, v_s, SV, v_full, v_empty, -1, pol, it, s, ph, [&](int i) {
                if ((i - seg.i0) % kP8ScaleChunk == 0 && i + kP8ScaleChunk < seg.i1) {
                    store_scales();                                     // of tiles i + 4 .. i + 7
                    fetch_scales(pos_of(i + 2 * kP8ScaleChunk), page_next);
                    page_next = page_of(pos_of(i + 3 * kP8ScaleChunk));
                }
            });
        }
        drain(v_full, SV, it, -1);
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
        // (with 32 rows, one thread a token and half of the rows)
        const int x = (warp >> 2) & 1, y = warp >> 3, w4 = warp & 3;
        const int bar = 1 + x + 2 * y;
        const int tok = threadIdx.x & 127;
        const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
        const uint32_t s_tm = lane_base + PS::kColS + x * PS::kNs + y * RH;
        const uint32_t o_tm = lane_base + PS::kColO + x * PS::kNp + y * RH;
        const uint32_t p_at = p_s + x * PS::kPBytes + tok * 16 + y * 2048;
        float* const my_ref = neg_ref + x * RP + y * RH;
        float4* const my_sum = sums + x * RP + y * RH;
        float2* const factor = factors + x * RP + y * RH;
        int* const my_max = warp_max + (x * PS::kParts + y) * 4 * (RH + 1);
        // Row r, column d of this part's O that a group hands over, in its own P
        // operand, which its last product has read.
        auto handed_at = [&](int group, int r, int d) -> float* {
            float* const base = handed + group * (PS::kPBytes / 4);
            if constexpr (PS::kParts == 1) return base + r * D + d;
            const int i = r * D + d;
            return base + ((i >> 9) * 2 + y) * 512 + (i & 511);
        };
        const int block_shift = min(p.page_shift, 6);
        uint32_t n_tiles = 0, n_merge = 0;       // phases of s_full and p_full, of m_full
        bool lent = false;                       // this group's P holds an O that it handed over
        int it0 = 0, sg = 0;                     // the CTA's tile number at the segment's start
        int chunk0 = 0;                          // and its chunk of scales
        // The product of this group's tile `it` has completed.
        auto wait_product = [&](int it) { all_wait(v_empty + 8 * (it % SV), it / SV); };
        while (walk.next(lens, seg)) {
            int b, rt;
            lens.split(seg.entry, b, rt);
            const int T = lens.tokens(b);
            const float4* scale4 = reinterpret_cast<const float4*>(row_scale + (sg & 1) * RP + y * RH);
            const int* lim = row_lim + (sg & 1) * RP + y * RH;
            const int lim_min =                                             // every row sees keys up to here
                T - p.sq + p.by_heads(rt * RP);
            const int first_i = seg.i0 + ((it0 & 1) != x ? 1 : 0);          // this group's first tile
            float l[RH];
            int ev = 0;
#pragma unroll
            for (int r = 0; r < RH; ++r) l[r] = 0.f;
            bool first = true;
            // Also keeps a group without a tile here from running ahead.
            all_wait(q_full + 8 * (sg & 1), sg >> 1);
            for (int i = first_i; i < seg.i1; i += 2) {
                const int it = it0 + i - seg.i0;
                const int pos = i * kP8Tokens + tok;
                const bool edge = (i + 1) * kP8Tokens - 1 > lim_min;        // some row does not see all of it

                all_wait(s_full + 8 * x, n_tiles);
                tc_fence_after();
                const float* sc = scale_ring + ((chunk0 + (i - seg.i0) / kP8ScaleChunk) % kP8ScaleChunks * kP8ScaleChunk +
                                                (i - seg.i0) % kP8ScaleChunk) * 16 + (tok >> block_shift);
                const float ks = sc[0];
                float vs = sc[8];
                // z = x - m, -inf where the row does not see the key.
                float sv[RH], z[RH];
                auto load_s = [&]() {
                    uint32_t h[RH], lo[RH];
                    if constexpr (RH == 8) {
                        uint32_t t[16];
                        tmem_ld16(s_tm, t);
#pragma unroll
                        for (int r = 0; r < 8; ++r) h[r] = t[r], lo[r] = t[8 + r];
                    } else {
                        tmem_ld16x2(s_tm, s_tm + RP, h, lo);
                    }
#pragma unroll
                    for (int r = 0; r < RH; r += 2) {
                        const float2 v = fma_x2(make_float2(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])),
                                                make_float2(0.0625f, 0.0625f),
                                                make_float2(__uint_as_float(h[r]), __uint_as_float(h[r + 1])));
                        sv[r] = v.x;
                        sv[r + 1] = v.y;
                    }
                };
                auto subtract_refs = [&]() {
#pragma unroll
                    for (int r = 0; r < RH; r += 4) {
                        const float4 f = scale4[r / 4];
                        const float4 m = *reinterpret_cast<const float4*>(my_ref + r);
                        const float2 kk = make_float2(ks, ks);
                        const float2 a = fma_x2(make_float2(sv[r], sv[r + 1]), mul_x2(make_float2(f.x, f.y), kk),
                                                make_float2(m.x, m.y));
                        const float2 c = fma_x2(make_float2(sv[r + 2], sv[r + 3]), mul_x2(make_float2(f.z, f.w), kk),
                                                make_float2(m.z, m.w));
                        z[r] = a.x;
                        z[r + 1] = a.y;
                        z[r + 2] = c.x;
                        z[r + 3] = c.y;
                    }
                    if (edge) {
#pragma unroll
                        for (int r = 0; r < RH; ++r)
                            if (pos > lim[r]) z[r] = -INFINITY;
                    }
                };
                load_s();
                subtract_refs();
                bool moves = first;
                {
                    float top = fmax3(z[0], z[1], z[2]);
#pragma unroll
                    for (int r = 3; r + 1 < RH; r += 2) top = fmax3(top, z[r], z[r + 1]);
                    top = fmaxf(top, z[RH - 1]);
                    // A NaN or infinite scale makes its block's values NaN.
                    if (!(fabsf(vs) <= 3.402823466e38f)) vs = __int_as_float(0x7fffffff);
                    moves |= top > kP8Slack || fabsf(vs) * pow2i(-ev) > kP8ScaleSlack;
                }
                if (named_any(bar, moves)) {
                    // Move the references: rows whose tile maximum is out of range.
                    // S is read again, so that it need not be kept above.
                    load_s();
                    float xs[RH];
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        xs[r] = sv[r] * (row_scale[(sg & 1) * RP + y * RH + r] * ks);
                        if (edge && pos > lim[r]) xs[r] = -INFINITY;
                    }
                    int mine = 0;
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        const int m = __reduce_max_sync(0xffffffffu, ordered(xs[r]));
                        if (lane == r) mine = m;
                    }
                    const uint32_t vb = __float_as_uint(fabsf(vs));
                    const uint32_t vtop = __reduce_max_sync(0xffffffffu, vb <= 0x7f7fffffu ? vb : 0u);
                    if (lane < RH) my_max[w4 * (RH + 1) + lane] = mine;
                    if (lane == 0) my_max[w4 * (RH + 1) + RH] = (int)vtop;
                    const float m_old = first || lane >= RH ? kP8Unseen : -my_ref[lane];
                    named_sync(bar, 128);
                    float m_new = m_old;
                    if (lane < RH) {
                        const float m = unordered(max(max(my_max[lane], my_max[RH + 1 + lane]),
                                                      max(my_max[2 * (RH + 1) + lane], my_max[3 * (RH + 1) + lane])));
                        if (m > m_old + kP8Slack) m_new = m;
                    }
                    const int vm = max(max(my_max[RH], my_max[2 * RH + 1]), max(my_max[3 * RH + 2], my_max[4 * RH + 3]));
                    // 2^-ev brings the largest scale to [0.5, 1); where it is below
                    // 2^-114 to 2^-13 at least, so that `unit` stays a normal number.
                    const int ev_top = min(max((vm >> 23) - 126, -113), 126);
                    const int ev_new = first || __int_as_float(vm) * pow2i(-ev) > kP8ScaleSlack ? ev_top : ev;
                    const float alpha = fast_exp2(m_old - m_new);
                    const float alpha_o = first ? 0.f : alpha * pow2i(max(ev - ev_new, -126));
                    if (w4 == 0 && lane < RH) my_ref[lane] = -m_new;
                    ev = ev_new;
#pragma unroll
                    for (int r = 0; r < RH; ++r) l[r] *= __shfl_sync(0xffffffffu, alpha, r);
                    if (!first) {
                        wait_product(it - 2);     // and so every product of this group so far
                        tc_fence_after();
#pragma unroll 1
                        for (int t = 0; t < kP8Terms; ++t) {
                            uint32_t o[RH];
                            tmem_ld_rows<RH>(o_tm + t * RP, o);
#pragma unroll
                            for (int k = 0; k < RH; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * __shfl_sync(0xffffffffu, alpha_o, k));
                            tmem_st_rows<RH>(o_tm + t * RP, o);
                        }
                        tmem_st_wait();
                    }
                    named_sync(bar, 128);
                    subtract_refs();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + 8 * x);
                if (edge) {
                    // Rows of V past the length may hold anything: zero them. A
                    // NaN code in a key that only some rows see would reach the
                    // others as 0 * NaN: its row is zeroed too, and the rows that
                    // see it are made NaN through P.
                    const int s = it % SV;
                    all_wait(v_full + 8 * s, it / SV);
                    const uint32_t at = v_s + s * TB + tok * D;
                    bool clear = pos >= T;
                    if (pos > lim_min && !clear) {
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
                    if constexpr (PS::kParts > 1) named_sync(5 + x, 256);   // both parts have looked
                    if (clear && y == 0)
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) st_shared_zero16(at + 16 * c);
                }
                const float vw = vs * pow2i(-ev) * kP8ProbScale;
                uint32_t packed[RH / 4][kP8Terms];       // a term of four rows
#pragma unroll
                for (int r = 0; r < RH; r += 4) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 pr = make_float2(fast_exp2(z[r + k]), fast_exp2(z[r + k + 1]));
                        const float2 sum = add_x2(make_float2(l[r + k], l[r + k + 1]), pr);
                        const float2 ww = mul_x2(pr, make_float2(vw, vw));
                        l[r + k] = sum.x;
                        l[r + k + 1] = sum.y;
                        w[k] = ww.x;
                        w[k + 1] = ww.y;
                    }
                    if (edge) {          // 0 * NaN: of a scale, or of a value that other rows see
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (z[r + k] == -INFINITY) w[k] = 0.f;
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
                if (lent) {                       // and handed-over O is read
                    all_wait(m_empty + 8 * y, n_merge + 1);
                    lent = false;
                }
                // Column term * RP + row; 16 columns of a token are 16 bytes.
                if constexpr (RH == 8) {
                    st_shared_v4(p_at, make_uint4(packed[0][0], packed[1][0], packed[0][1], packed[1][1]));
                    st_shared_v4(p_at + 2048, make_uint4(packed[0][2], packed[1][2], packed[0][3], packed[1][3]));
                } else {
#pragma unroll
                    for (int t = 0; t < kP8Terms; ++t)
                        st_shared_v4(p_at + t * (RP / 16) * 2048,
                                     make_uint4(packed[0][t], packed[1][t], packed[2][t], packed[3][t]));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * x);
                ++n_tiles;
                first = false;
            }

            // ------------------------------------------------ end of a segment
            const int len = seg.i1 - seg.i0;
            const int cnt0 = (len + ((it0 & 1) == 0 ? 1 : 0)) / 2, cnt1 = len - cnt0;
            const bool both = cnt0 > 0 && cnt1 > 0;
            if ((x ? cnt1 : cnt0) > 0) {
                const float sum = reduce_rows<RH>(l, lane);
                if (lane < RH) reinterpret_cast<float*>(my_sum + lane)[w4] = sum;
                named_sync(bar, 128);
                const bool whole = seg.i0 == 0 && seg.i1 == seg.n;
                int c0 = 0, n = 1;                // the CTAs that share the unit
                if (!whole) plan_s->sharers(seg, c0, n);
                // This group's last tile is the segment's last or the one before.
                const int last = it0 + len - 1;
                wait_product((last & 1) == x ? last : last - 1);
                tc_fence_after();
                float o[RH];
#pragma unroll
                for (int r = 0; r < RH; ++r) o[r] = 0.f;
                // In units of the values; a row's factor comes later, times which this
                // could fall below the normal numbers.
                float unit = pow2i(ev) * (1.f / kP8ProbScale);
#pragma unroll
                for (int t = 0; t < kP8Terms; ++t) {
                    uint32_t u[RH];
                    tmem_ld_rows<RH>(o_tm + t * RP, u);
#pragma unroll
                    for (int r = 0; r < RH; ++r) o[r] = fmaf(__uint_as_float(u[r]), unit, o[r]);
                    unit *= 1.f / kP8TermStep;
                }
                tc_fence_before();
                // D = 64 products keep 16 of their rows in each warp's 32 lanes.
                const bool mine = D == 128 || lane < 16;
                const int dim = D == 128 ? tok : w4 * 16 + lane;
                // Of two groups, the one without the last tile hands its O over.
                if (both && x != (last & 1)) {
#pragma unroll
                    for (int r = 0; r < RH; ++r)
                        if (mine) *handed_at(x, r, dim) = o[r];
                    if (tok < RH) {
                        const float4 q = my_sum[tok];
                        other[y * RH + tok] = make_float2(-my_ref[tok], q.x + q.y + q.z + q.w);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(m_full + 8 * y);
                    ++n_merge;
                    lent = true;
                } else {
                    if (both) all_wait(m_full + 8 * y, n_merge);
                    const size_t slot_floats = p8_slot_floats(RP, D);
                    float* slot = p.part + ((size_t)blockIdx.x * 2 + (seg.i0 == 0 ? 1 : 0)) * slot_floats;
                    const int* rows_out = row_out + (sg & 1) * RP + y * RH;
                    if (tok < RH) {
                        const float4 q = my_sum[tok];
                        float m = -my_ref[tok], ls = q.x + q.y + q.z + q.w, a0 = 1.f, a1 = 0.f;
                        if (both) {
                            const float2 u = other[y * RH + tok];
                            const float top = fmaxf(m, u.x);
                            a0 = fast_exp2(m - top);
                            a1 = fast_exp2(u.x - top);
                            m = top;
                            ls = ls * a0 + u.y * a1;
                        }
                        if (whole) {
                            const bool some = ls > 0.f || ls != ls;
                            const float inv = some ? __fdividef(1.f, ls) : 0.f;
                            a0 *= inv;
                            a1 *= inv;
                            if (p.lse && rows_out[tok] >= 0)
                                p.lse[rows_out[tok]] = some ? (m + __log2f(ls)) * 0.6931471805599453f : -INFINITY;
                        } else {
                            slot[RP * D + y * RH + tok] = m;
                            slot[RP * D + RP + y * RH + tok] = ls;
                        }
                        factor[tok] = make_float2(a0, a1);
                    }
                    named_sync(bar, 128);
                    // With up to 16 rows whole outputs are gathered in the group's own
                    // P operand, whose last product has read it, for 16-byte stores
                    // from a short loop: what runs once per unit costs its
                    // instructions' fetch (8 rows, 128 x 4096 tokens: 25.7 -> 25.5 us).
                    // With 32 rows that lost to 2-byte stores (registers).
                    constexpr bool kGather = PS::kParts == 1;
                    float* const own = handed + x * (PS::kPBytes / 4);
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        const float2 f = factor[r];
                        float v = o[r] * f.x;
                        if (both && mine) v = fmaf(*handed_at(x ^ 1, r, dim), f.y, v);
                        if (!mine) continue;
                        if (!whole)
                            slot[(y * RH + r) * D + dim] = v;
                        else if (kGather)
                            own[r * D + dim] = v;
                        else if (rows_out[r] >= 0)
                            p.out[(size_t)rows_out[r] * D + dim] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
                    }
                    if (both) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(m_empty + 8 * y);
                        ++n_merge;
                    }
                    if (kGather && whole) {
                        named_sync(bar, 128);
#pragma unroll 1
                        for (int item = tok; item < RH * D / 8; item += 128) {
                            const int r = item / (D / 8);
                            const float4* from = reinterpret_cast<const float4*>(own + item * 8);
                            const float4 a = from[0], c = from[1];
                            if (rows_out[r] >= 0)
                                *reinterpret_cast<uint4*>(p.out + (size_t)rows_out[r] * D + item % (D / 8) * 8) =
                                    make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(c.x, c.y),
                                               pack_bf16x2(c.z, c.w));
                        }
                    }
                    if (!whole) {
                        // The last of the unit's CTAs to arrive merges it:
                        //   M = max m_c, L = sum l_c 2^(m_c - M), O = sum O_c 2^(m_c - M) / L.
                        named_sync(bar, 128);
                        if (tok == 0)             // releases the group's stores, which the barrier ordered before
                            last_flag[bar - 1] = arrive_last(p.counters + (size_t)c0 * PS::kParts + y, p.tag, n);
                        named_sync(bar, 128);
                        if (last_flag[bar - 1]) {
                            p8_merge<D, RP, RH>(p, c0, n, y * RH, tok, rows_out);
                        }
                    }
                }
                // The sums and references are read before the next segment writes them.
                named_sync(bar, 128);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty + 8 * (sg & 1));
            if (!kLoaderSplits && x != ((it0 + len - 1) & 1) && y * 4 + w4 < RP / 8) {
                P8Walk<RP> peek = walk;
                if (peek.next(lens, seg)) {
                    lens.split(seg.entry, b, rt);
                    const QRows q = load_rows(b, rt, seg.g, (y * 4 + w4) * 8);
                    all_wait(q_empty + 8 * ((sg + 1) & 1), ((sg + 1) >> 1) + 1);
                    split_rows(q, lens.tokens(b), (sg + 1) & 1, (y * 4 + w4) * 8);
                }
            }
            it0 += len;
            chunk0 += (len + kP8ScaleChunk - 1) / kP8ScaleChunk;
            ++sg;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == SW + 1) tmem_dealloc(tmem, PS::kTmemCols);
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
    cfg.blockDim = dim3(PS::kThreads);
    cfg.dynamicSmemBytes = PS::kSmemBytes;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gqa_paged_fp8_kernel<D, RP>, a.tm_k, a.tm_v, a.p);
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
