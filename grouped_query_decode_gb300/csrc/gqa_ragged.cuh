// Causal attention of packed batches (whole prompts, or chunks over a paged
// cache) on the 5th-generation tensor cores, for sm_103a.
//
// A unit is (sequence, KV head, 2 * tq new tokens), tq = floor(128 / (H / G)): two
// 128-row tiles A and B whose rows are the tokens' heads that read the KV head,
// token by token, so K and V are read once for all of them. Per key tile of 128:
//     S_X = Q_X K^T     M = 128, N = 128, K = D     (A, B operands in shared memory)
//     O_X += P_X V      M = 128, N = D,   K = 128   (P in tensor memory)
// with a running reference m per row that moves to the maximum only when 64 weights
// of a tile sum to more than 2^8 (then O_X is rescaled in tensor memory), fp32 sums,
// and P rounded to bf16 over the columns of S_X that it came from. So a tile's scores
// are read once and no maximum is taken (with one, and a weight above 2^8 as the sign,
// the prompt of 16384 below took 1444 us for 1421).
//
// Work: gqa_ragged_plan.cuh. One CTA per SM walks the units of its share; parts
// of units that shares cut leave (O, m, l) in the workspace, and the CTA that
// arrives last merges them in the order of the parts.
//
// Warps: 0-7 and 8-15 softmax of A and B, two threads per row, 64 keys of a tile
// each; 16-19 outputs; 20 issues the products, always one of A, one of B, so that
// each tile's softmax runs behind the other's products; 21 loads Q and K by TMA, a
// lane per page, 22 V, of which it mends the tiles that reach past the first row's
// limit; 23 plans and hands the units out through a ring in shared memory. Every
// wait is bounded; after one has expired the CTA runs through its units without
// work, so that the counters end at zero.
//
// Rounding: P to bf16, as the products take it (at most 2^-8 of each weight; out
// differs from the formula in 64 bits by 2.0e-3 to 2.4e-3 of its norm, out rounded to
// bf16 alone by 1.5e-3 to 1.7e-3), and out to bf16, once. Scores, m, l, O and the parts are fp32.
//
// V at positions that only some rows see: a masked key's weight is 0, and 0 times
// NaN or infinity is not. In tiles past the first row's limit warp 22 zeroes what
// no row sees, and takes out values that are not finite; a row that sees such a
// value gets NaN in its column with the output.
//
// What bounds it, on one GB300 (copy 6.79 TB/s, bf16 products 1879 TFLOP/s):
// - long prompts: 16384 tokens, 32/8 heads, D 128 take 1420 us back to back (the power
//   cap holds the clock down) and 1296 us in a burst, 1.70 PFLOP/s; the products alone
//   are 1171 us. Without its softmax an earlier form took 1100 us, without its products
//   1120: both are nearly full, and what is left is their handing over to each other,
//   some 450 of a step's 2900 cycles (a step: one key tile with both row tiles).
// - single tokens: HBM (64 sequences of up to 16384 keys 386 us, 6.6 TB/s).
// - D 64: the softmax's chain. A step's products are 1024 cycles, but scores, weights and
//   the next scores follow one another, and a step takes 2800, as with D 128 (the long
//   prompt 1192 us, 585 at the roofline; 24 ragged ones 286, 110 at the roofline).
// - short sequences: 2 to 3 us at a unit's start and end, 4 us before a launch's first
//   scores, 4 to 15 us for a merge (8 prompts of 1024, 16 heads, D 64 41 us, 10 at
//   the roofline; 64 single tokens of 1024 keys, D 64, 42, 20 at the roofline; chunks
//   among single tokens 260 to 290 us by the order of the sequences, 146 at the roofline).
//
// Why this split of the warps: one softmax thread per row held 128 scores, and the 8
// prompts took 54 us for 48 with two; one pipeline for units with one row tile, and
// one warp that loaded K and V both and mended V between, took 475 us for the single
// tokens' 381.
#pragma once

#include <atomic>

#include "gqa_device.cuh"
#include "gqa_paged_fp8.cuh"
#include "gqa_ragged.h"
#include "gqa_ragged_plan.cuh"
#include "tcgen05.cuh"

namespace gqa {

constexpr int kRgThreads = 768;
constexpr int kRgOut = 16, kRgMma = 20, kRgLoadK = 21, kRgLoadV = 22, kRgPlan = 23;   // first warps of the roles
constexpr float kRgSlack = 256.0f;       // sum of 64 weights at which the reference moves
constexpr uint64_t kRgTileNs = 16000;    // what a key tile may take at most (it takes 1600)

template <int D>
struct RgShape {
    static constexpr int kBlock = 128 * 128;              // 128 rows x 128 B, 128-byte swizzle
    static constexpr int kBlocks = D / 64;
    static constexpr int kTile = kBlocks * kBlock;        // Q, K or V of one tile
    // K and V tiles in rings of their own, each filled by a warp of its own.
    static constexpr int kStagesK = D == 128 ? 2 : 5, kStagesV = D == 128 ? 2 : 5, kStages = kStagesK + kStagesV;
    static constexpr int kMlBytes = 2 * 128 * (8 + 8 + 4);
    static constexpr int kUnitBytes = kRgUnits * 64;
    static constexpr int kTodo = 128 + kRgThreads / 32 * 8;      // behind the warps' sums
    static constexpr int kMiscBytes = kTodo + 2 * 64;
    static constexpr int kBars = 3 * kStages + 2 * 10 + 2 * kRgUnits + 3;
    static constexpr int kSmemBytes =
        2 * kTile + kStages * kTile + kMlBytes + kUnitBytes + kMiscBytes + 8 * kBars;
    // Columns: S_A | S_B | O_A | O_B, with P over S, that of each 64 keys over the first
    // half of their scores; D = 64 has room for P apart (S_A | S_B | P_A | P_B | O_A |
    // O_B), so that the next scores wait only until these have been read.
    static constexpr bool kApart = D == 64;
    static constexpr uint32_t kColS = 0, kColP = kApart ? 256 : 0, kStepP = kApart ? 64 : 128, kColO = kApart ? 384 : 256;
    static constexpr uint32_t kHalfP = kApart ? 32 : 64;  // columns from the weights of the first 64 keys to the others'
    static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");
    static_assert(16 + 4 * kRgUnits <= 64 && kTodo % 16 == 0, "flags of units; units as 16-byte words");
    static_assert((2 + kStages) * kTile >= 25 * 1024 + 2 * 160 * D * 4 + 256, "a merge's weights, and a row of 160 parts twice");
};

// Eight words to 32-byte aligned memory, or to 16-byte aligned.
__device__ __forceinline__ void store32(void* to, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ void load_scores(uint32_t from, uint32_t (&s)[16]) { tmem_ld16(from, s); }
__device__ __forceinline__ void load_scores(uint32_t from, uint32_t (&s)[32]) { tmem_ld32(from, s); }

// Hides the scores from `see` + 1 on.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&s)[N], int see) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = i <= see ? s[i] : 0xff800000u;
}

// Weights 2^(s * scale + neg), in pairs of bf16, and their sums.
template <int N>
__device__ __forceinline__ void weigh(const uint32_t (&s)[N], float2 scale, float2 neg, float2 (&sum)[2], uint32_t* w) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 z = fma_x2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), scale, neg);
        const float2 e = make_float2(fast_exp2(z.x), fast_exp2(z.y));
        sum[(i / 2) & 1] = add_x2(sum[(i / 2) & 1], e);
        w[i / 2] = pack_bf16x2(e.x, e.y);
    }
}

// Whether any of a named barrier's 64 threads votes.
__device__ __forceinline__ bool pair_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0;
}

// A unit with rows in tile A alone: its key tiles go to both pipelines in turn, so
// that one tile's softmax runs behind the other's products; their two O are joined
// with the output. Key tile of pipeline x's j-th step, and steps of pipeline x:
struct RgSteps {
    bool dual;
    int a, b;
    __device__ __forceinline__ explicit RgSteps(const RgUnit& u) {
        dual = u.tokens[1] == 0 && u.tiles[0] > 1;
        a = dual ? (u.tiles[0] + 1) / 2 : u.tiles[0];
        b = dual ? u.tiles[0] / 2 : u.tiles[1];
    }
};

__device__ __forceinline__ RgSeq rg_sequence(const RaggedParams& p, int b) {
    RgSeq s = {0, 0, 0};
    if (b < p.B) {
        s.start = clamp_len(__ldg(p.cu + b), p.N);
        s.n = max(min(__ldg(p.cu + b + 1), p.N), s.start) - s.start;
        s.T = p.table ? clamp_len(__ldg(p.lens + b), p.max_pages << p.page_shift) : s.n;
    }
    return s;
}

// What a wait does when its phase has not completed yet: out of line, because
// instruction fetches are what short units wait for.
static __device__ __noinline__ bool rg_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status,
                                          uint64_t tmo) {
    return wait_phase(bar, parity, abort_flag, status, tmo);
}
static __device__ __noinline__ bool rg_wait_longer(uint32_t bar, uint32_t parity, uint64_t limit) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > limit) return false;
    return true;
}

// 1-D copy into shared memory, completing bytes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Merges the parts of a unit with all threads of the CTA: M = max m, w = 2^(m - M),
// L = sum l w, O = sum O w / L, part by part in their order. All parts of a block of
// rows come into one half of `room` while the block before is summed from the other.
// This runs once or twice per CTA, so its time is latency and instruction fetches:
// loops are short. `bars`: two barriers, whose phases are bits of `phases`.
constexpr uint32_t kRgWeightBytes = 24 * 1024;
template <int D>
__device__ __forceinline__ void rg_merge(const RaggedParams& p, const RgUnit& u, unsigned char* room, uint32_t room_bytes,
                                         uint32_t bars, uint32_t& phases) {
    constexpr int kChunks = D / 4;
    const int n = u.parts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows_a = u.tokens[0] * p.heads_per_group, rows_all = rows_a + u.tokens[1] * p.heads_per_group;
    float* const inverse = reinterpret_cast<float*>(room);        // [256]
    float2* const weights = reinterpret_cast<float2*>(inverse + 256);   // [rows][n]: (m, l), then w in x
    unsigned char* const held = room + 1024 + kRgWeightBytes;     // O of the parts, [n][rows][D], twice
    const uint32_t half = (room_bytes - 1024 - kRgWeightBytes) / 2 & ~127u;
    const int block = half / (n * D * 4), most = min(rows_all, (int)(kRgWeightBytes / (8 * n)));
    // The first part's slot is its counter's; later ones continue from the CTA before.
    auto part = [&](int i) { return p.part + (size_t)(i == 0 ? u.counter : 2 * (u.first + i)) * rg_slot_floats(D); };
    // Rows count A's, then B's.
    auto slot_row = [&](int r) { return r < rows_a ? r : 128 + r - rows_a; };
    auto out_row = [&](int r) {
        const int x = r >= rows_a, in = x ? r - rows_a : r, tok = p.by_heads(in);
        return (size_t)(u.row0 + x * p.tq + tok) * p.H + (size_t)u.g * p.heads_per_group + (in - tok * p.heads_per_group);
    };
    asm volatile("fence.proxy.async;" ::: "memory");              // the parts were written by plain stores
#pragma unroll 1
    for (int w0 = 0; w0 < rows_all; w0 += most) {
        const int w1 = min(rows_all, w0 + most);
        auto end_of = [&](int r) { return min(min(r + block, w1), r < rows_a ? rows_a : rows_all); };   // of r's block
        auto fetch = [&](int r, int b) {                          // by the last warp
            const uint32_t bytes = (end_of(r) - r) * D * 4;
            if (lane == 0) mbar_arrive_expect_tx(bars + 8 * b, n * bytes);
            __syncwarp();
#pragma unroll 1
            for (int i = lane; i < n; i += 32)
                bulk_load(smem_addr(held) + b * half + i * bytes, part(i) + (size_t)slot_row(r) * D, bytes, bars + 8 * b);
        };
        const bool feeds = warp == kRgThreads / 32 - 1;
        if (feeds) fetch(w0, 0);
#pragma unroll 2
        for (int e = threadIdx.x; e < (w1 - w0) * n; e += kRgThreads) {
            const int r = e / n, s = 256 * D + slot_row(w0 + r);
            const float* const from = part(e - r * n);
            weights[e] = make_float2(__ldcg(from + s), __ldcg(from + s + 256));
        }
        __syncthreads();
#pragma unroll 1
        for (int r = w0 + (int)threadIdx.x; r < w1; r += kRgThreads) {
            float2* const mine = weights + (r - w0) * n;
            float M = -INFINITY, L = 0.f;
#pragma unroll 2
            for (int i = 0; i < n; ++i) M = fmaxf(M, mine[i].x);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const float l = mine[i].y, w = l == 0.f ? 0.f : fast_exp2(mine[i].x - M);
                mine[i].x = w;
                L += l * w;
            }
            inverse[r - w0] = L == 0.f ? 0.f : 1.f / L;
            if (p.lse) p.lse[out_row(r)] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        }
        __syncthreads();
        int b = 0;
#pragma unroll 1
        for (int r0 = w0; r0 < w1; b ^= 1) {
            const int r1 = end_of(r0);
            if (feeds && r1 < w1) fetch(r1, b ^ 1);
            if (!rg_wait_longer(bars + 8 * b, phases >> b & 1, p.wait_timeout_ns)) atomicOr(p.status, kStatusTimeout);
            phases ^= 1u << b;
            const float4* const o = reinterpret_cast<const float4*>(held + b * half);
            const int items = (r1 - r0) * kChunks;
#pragma unroll 1
            for (int item = threadIdx.x; item < items; item += kRgThreads) {
                const int r = r0 + item / kChunks;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int i = 0; i < n; ++i) {
                    const float w = weights[(r - w0) * n + i].x;
                    const float4 v = o[i * items + item];                  // 0 of it, too, keeps a NaN
                    y.x = fmaf(v.x, w, y.x);
                    y.y = fmaf(v.y, w, y.y);
                    y.z = fmaf(v.z, w, y.z);
                    y.w = fmaf(v.w, w, y.w);
                }
                const float f = inverse[r - w0];
                *(reinterpret_cast<uint2*>(p.out + out_row(r) * D) + item % kChunks) =
                    make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
            }
            __syncthreads();
            r0 = r1;
        }
    }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kRgThreads, 1)
    gqa_ragged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ RaggedParams p) {
    using RS = RgShape<D>;
    constexpr int S = RS::kStages, SK = RS::kStagesK, SV = RS::kStagesV;       // V's stages follow K's
    constexpr uint32_t kBlock = RS::kBlock, kTile = RS::kTile;

    extern __shared__ __align__(1024) unsigned char smem_raw[];
    // There is no static shared memory, so that the dynamic one starts on the 1024
    // bytes of the swizzle atom.
    const uint32_t raw = smem_addr(smem_raw);
    if (raw & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }
    const uint32_t q_s = raw, ring_s = q_s + 2 * kTile;
    unsigned char* gen = smem_raw + (2 + S) * kTile;
    float2* const ml = reinterpret_cast<float2*>(gen);               // [2][128]
    float* const top_s = reinterpret_cast<float*>(gen + 2048);       // [2][2][128]: maxima of each half of a tile
    float* const sum_s = reinterpret_cast<float*>(gen + 4096);       // [2][128]: sums of the second halves
    gen += RS::kMlBytes;
    // Per column the first position of a value that is not finite, in the workspace:
    // it is hardly ever touched.
    int* const bad = p.bad + (size_t)blockIdx.x * kRgUnits * D;      // [units][D]
    RgUnit* const units = reinterpret_cast<RgUnit*>(gen);
    gen += RS::kUnitBytes;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gen);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(gen + 4);
    volatile int* const todos = reinterpret_cast<volatile int*>(gen + 8);
    int* const bad_flag = reinterpret_cast<int*>(gen + 16);          // [units]
    long long* const first_s = reinterpret_cast<long long*>(gen + 64);   // [1], [2]: sequence and offset of the share's start
    RgShares* const shares = reinterpret_cast<RgShares*>(gen + 96);
    long long* const warp_sum = reinterpret_cast<long long*>(gen + 128); // [warps]
    RgUnit* const todo = reinterpret_cast<RgUnit*>(gen + RS::kTodo);     // [2]: units to merge
    gen += RS::kMiscBytes;
    const uint32_t full = smem_addr(gen), empty = full + 8 * S, mended = empty + 8 * S;
    const uint32_t q_full = mended + 8 * S, q_empty = q_full + 16, s_full = q_empty + 16, p_full = s_full + 16;
    const uint32_t s_free = p_full + 16, pv_done = s_free + 16;
    const uint32_t o_full = pv_done + 16, o_empty = o_full + 16, ml_full = o_empty + 16, fin = ml_full + 16;
    const uint32_t u_full = fin + 8, u_empty = u_full + 8 * kRgUnits, merge_bar = u_empty + 8 * kRgUnits;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = p.wait_timeout_ns;

    // Barriers, by threads of several warps.
    if (warp == 0 && lane < S) {
        mbar_init(full + 8 * lane, 1);
        mbar_init(empty + 8 * lane, 1);
        mbar_init(mended + 8 * lane, 1);
        fence_barrier_init();
    } else if (warp == 1 && lane < 2) {
        mbar_init(q_full + 8 * lane, 1);
        mbar_init(q_empty + 8 * lane, 1);
        mbar_init(s_full + 8 * lane, 1);
        mbar_init(p_full + 8 * lane, 8);
        mbar_init(s_free + 8 * lane, 8);
        mbar_init(pv_done + 8 * lane, 1);
        mbar_init(o_full + 8 * lane, 1);
        mbar_init(o_empty + 8 * lane, 4);
        mbar_init(ml_full + 8 * lane, 4);
        mbar_init(merge_bar + 8 * lane, 1);
        fence_barrier_init();
    } else if (warp == 2 && lane < kRgUnits) {
        mbar_init(u_full + 8 * lane, 1);
        mbar_init(u_empty + 8 * lane, 23);        // softmax and output warps, products, loads
        bad_flag[lane] = 0;
        fence_barrier_init();
    } else if (warp == 3 && lane == 0) {
        mbar_init(fin, 1);
        *abort_flag = 0;
        *todos = 0;
        first_s[1] = p.B;
        fence_barrier_init();
    }
    if (warp == kRgMma) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == kRgLoadK && lane < 3) tma_prefetch_desc(lane == 0 ? &tm_q : lane == 1 ? &tm_k : &tm_v);
    pdl_launch_dependents();
    pdl_wait_primary();

    // The line's length, and the sequence in which this CTA's share starts. With few
    // sequences the planning warp finds them by itself, below, and the others' start
    // does not wait for it (a tiny prompt 13.1 -> 11.2 us); with more, every thread takes
    // some in a row.
    const RgLine line = RgLine::of(p.tq, p.G, D);
    const bool few = p.B <= 128;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!few) {
        const int per = (p.B + kRgThreads - 1) / kRgThreads;
        const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
        long long mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) mine += line.head(rg_sequence(p, b)) * p.G;
        long long sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll 4
        for (int w = 0; w < kRgThreads / 32; ++w) {
            const long long y = warp_sum[w];
            if (w < warp) before += y;
            total += y;
        }
        long long at = before + sum - mine;
        if (threadIdx.x == 0) *shares = RgShares::of(total, gridDim.x);
        __syncthreads();
        const RgShares sh = *shares;
        const long long from = (int)blockIdx.x < sh.ctas ? sh.at(blockIdx.x) : total;
        if (at <= from && from < at + mine)
#pragma unroll 1
            for (int b = b0; b < b1; ++b) {
                const long long y = line.head(rg_sequence(p, b)) * p.G;
                if (from < at + y) {
                    first_s[1] = b;
                    first_s[2] = at;
                    break;
                }
                at += y;
            }
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](uint32_t bar, uint32_t parity, uint64_t more = 0) {
        return mbar_try_wait(bar, parity & 1) || rg_wait_slow(bar, parity & 1, abort_flag, p.status, tmo + more);
    };
    // The next unit, for every lane of a warp. Waits on although the CTA has given
    // up its work: units keep coming, as long as the longest of them may take (69 s: 2^31
    // keys are 25). False: none comes any more.
    auto next_unit = [&](uint32_t n) {
        const uint32_t bar = u_full + 8 * (n % kRgUnits), parity = (n / kRgUnits) & 1;
        return mbar_try_wait(bar, parity) || rg_wait_longer(bar, parity, 8 * tmo + (1ull << 36));
    };

    if (warp >= kRgMma) {
        if (warp == kRgPlan) {
            // ------------------------------------------------------------ plan
            // Sequence b, whose units start at `at` on the line, KV head g, pair pr.
            const int c = blockIdx.x;
            if (few) {
                long long total = 0;
#pragma unroll 4
                for (int b = lane; b < 128; b += 32) total += line.head(rg_sequence(p, b)) * p.G;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                const RgShares sh = RgShares::of(total, gridDim.x);
                const long long from = c < sh.ctas ? sh.at(c) : total;
                long long at = 0;
#pragma unroll 1
                for (int b = 0; b < p.B; b += 32) {
                    const long long y = line.head(rg_sequence(p, b + lane)) * p.G;
                    long long sum = y;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long z = __shfl_up_sync(0xffffffffu, sum, o);
                        if (lane >= o) sum += z;
                    }
                    if (at + sum - y <= from && from < at + sum) {
                        first_s[1] = b + lane;
                        first_s[2] = at + sum - y;
                    }
                    at += __shfl_sync(0xffffffffu, sum, 31);
                }
                if (lane == 0) *shares = sh;
                __syncwarp();
            }
            const RgShares sh = *shares;
            const long long to = c < sh.ctas ? sh.at(c + 1) : 0;
            int b = (int)first_s[1], g = 0, pr = 0, pairs = 0;
            long long at = first_s[2], head = 0;
            int chunk = b;                          // lanes hold sequences chunk + lane
            RgSeq mine = rg_sequence(p, chunk + lane), seq = {0, 0, 0};
            bool inside = false, first = true;
            auto plan = [&](RgUnit& u) {            // the next unit with a part for this CTA
                while (true) {
                    if (!inside) {
                        for (; b < p.B && at < to; ++b) {
                            if (b >= chunk + 32) {
                                chunk = b;
                                mine = rg_sequence(p, chunk + lane);
                            }
                            seq.n = __shfl_sync(0xffffffffu, mine.n, b - chunk);
                            if (seq.n > 0) break;
                        }
                        if (b >= p.B || at >= to) return false;
                        seq.start = __shfl_sync(0xffffffffu, mine.start, b - chunk);
                        seq.T = __shfl_sync(0xffffffffu, mine.T, b - chunk);
                        pairs = line.pairs(seq.n);
                        head = line.head(seq);
                        g = pr = 0;
                        if (first) {
                            const long long y = sh.at(c) - at;
                            g = min((int)((float)y / (float)head), p.G - 1);       // or the one beside it
                            while (g * head > y) --g;
                            while ((g + 1) * head <= y) ++g;
                            pr = line.pair_at(seq, y - g * head);
                        }
                        first = false;
                        inside = true;
                    }
                    if (pr == pairs) {
                        pr = 0;
                        if (++g == p.G) {
                            at += head * p.G;
                            ++b;
                            inside = false;
                            continue;
                        }
                    }
                    const long long unit = at + g * head + line.start(seq, pr);
                    if (unit >= to) return false;
                    u.seq = b;
                    u.g = g;
                    if (rg_unit(line, sh, c, seq, pr++, unit, &u)) return true;
                }
            };
            bool more = true;
            int longest = 0;                        // unit, in key tiles
            for (uint32_t n = 0; more; ++n) {
                RgUnit u;
                more = plan(u);
                u.valid = more;                     // the last one handed out ends the list
                if (lane == 0) {
                    if (more && u.slot >= 0) tag_counter(p.counters + u.counter, p.tag);
                    if (!rg_wait_longer(u_empty + 8 * (n % kRgUnits), ((n / kRgUnits) & 1) ^ 1,
                                        4 * tmo + kRgUnits * kRgTileNs * longest)) {
                        *abort_flag = 1;
                        atomicOr(p.status, kStatusTimeout);
                    }
                    if (more) longest = max(longest, max(u.tiles[0], u.tiles[1]));
                    units[n % kRgUnits] = u;
                    mbar_arrive(u_full + 8 * (n % kRgUnits));
                }
                __syncwarp();
            }
        } else if (warp >= kRgLoadK) {
            // --------------------- loads: Q and K by one warp, V by another, which mends it
            const bool v_warp = warp == kRgLoadV;
            const int page_rows = PAGED ? min(1 << p.page_shift, kRgTile) : kRgTile;
            const int boxes = kRgTile / page_rows;
            const CUtensorMap* const tm = v_warp ? &tm_v : &tm_k;
            const uint32_t stages = v_warp ? SV : SK, stage0 = v_warp ? SK : 0;
            uint32_t stage = 0, turn = 0, nq = 0;    // stage of the ring, its parity; phases of Q_x in bit x
            // Copies issued: bit s, bit 16 + x; and the parity of the last of each.
            uint32_t issued = 0, parity = 0;
            auto note = [&](int bit, uint32_t phase) {
                issued |= 1u << bit;
                parity = (parity & ~(1u << bit)) | ((phase & 1) << bit);
            };
            for (uint32_t n = 0; next_unit(n); ++n) {
                __syncwarp();
                const RgUnit& u = units[n % kRgUnits];
                if (!u.valid) break;
                const int all = max(u.tiles[0], u.tiles[1]), last = u.pos_last, ug = u.g, lim = u.pos0;
                bool any_bad = false;
                if (!v_warp) {
                    const bool dual = RgSteps(u).dual;       // both pipelines have tile A's rows
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        if ((x ? u.tiles[1] : u.tiles[0]) == 0 && !dual) continue;
                        const bool ok = !*abort_flag && wait(q_empty + 8 * x, (nq >> x) ^ 1);
                        if (ok) note(16 + x, nq >> x);
                        nq ^= 1u << x;
                        if (ok && lane == 0) {
                            mbar_arrive_expect_tx(q_full + 8 * x, RS::kBlocks * p.tq * p.heads_per_group * 128);
#pragma unroll
                            for (int k = 0; k < RS::kBlocks; ++k)
                                tma_load_3d(q_s + x * kTile + k * kBlock, &tm_q, q_full + 8 * x, k * 64,
                                            ug * p.heads_per_group, u.row0 + (dual ? 0 : x * p.tq));
                        }
                    }
                }
                // This lane's page of key tile j: its slab, or the one past the last.
                auto slab = [&](int j) {
                    int page = p.num_pages;
                    if (lane < boxes) {
                        const int t = (u.j0 + j) * kRgTile + lane * page_rows;
                        if (t <= last) {
                            const int e = __ldg(p.table + (size_t)u.seq * p.max_pages + (t >> p.page_shift));
                            if ((unsigned)e < (unsigned)p.num_pages) page = e;
                        }
                    }
                    return page == p.num_pages ? p.num_pages * p.G : page * p.G + ug;
                };
                int now = 0;
                // With V, step j issues tile j and then sees tile j - 1 land, before the
                // next copy goes to that one's stage.
#pragma unroll 1
                for (int j = 0; j < all + v_warp; ++j) {
                    const int t0 = (u.j0 + j) * kRgTile;
                    if (j < all) {
                        if (PAGED && j == 0) now = slab(0);
                        const int then = PAGED && j + 1 < all ? slab(j + 1) : 0;
                        const uint32_t s = stage0 + stage, bar = full + 8 * s;
                        bool ok = !*abort_flag && wait(empty + 8 * s, turn ^ 1);
                        ok = __all_sync(0xffffffffu, ok);
                        if (ok && !(blockIdx.x == 0 && !v_warp && n == 0 && j == p.skip_tile)) {     // injected fault
                            note(s, turn);
                            if (lane == 0) mbar_arrive_expect_tx(bar, kTile);
                            __syncwarp();
                            const uint32_t dst = ring_s + s * kTile + lane * page_rows * 128;
                            if (lane < boxes)
#pragma unroll
                                for (int k = 0; k < RS::kBlocks; ++k) {
                                    if (PAGED)
                                        tma_load_3d(dst + k * kBlock, tm, bar, k * 64,
                                                    boxes > 1 ? 0 : t0 & ((1 << p.page_shift) - 1), now);
                                    else
                                        tma_load_3d(dst + k * kBlock, tm, bar, k * 64, ug, u.key0 + t0);
                                }
                        }
                        now = then;
                    }
                    // The tile before: its stage, and the parity of its turn.
                    const uint32_t s = stage0 + (stage == 0 ? stages : stage) - 1, was = stage == 0 ? turn ^ 1 : turn;
                    if (j < all && ++stage == stages) {
                        stage = 0;
                        turn ^= 1;
                    }
                    if (!v_warp || j == 0) continue;
                    const int t1 = t0 - kRgTile;
                    const uint32_t v_s = ring_s + s * kTile;
                    const bool ok = !*abort_flag && wait(full + 8 * s, was);
                    if (!__all_sync(0xffffffffu, ok) || t1 + kRgTile - 1 <= lim) continue;
                    // Rows [r0, r1) are seen by some, those from r1 on by none.
                    const int r0 = max(0, lim + 1 - t1), r1 = max(0, min(kRgTile, last + 1 - t1));
                    auto chunk = [&](int r, int c) { return v_s + (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
                    constexpr int kChunks = D / 8;
#pragma unroll 1
                    for (int i = r1 * kChunks + lane; i < kRgTile * kChunks; i += 32)
                        st_shared_zero16(chunk(i / kChunks, i % kChunks));
                    // x * 0 is NaN for what is not finite.
                    uint32_t sum = 0;
                    const uint32_t zero = 0;
#pragma unroll 2
                    for (int i = r0 * kChunks + lane; i < r1 * kChunks; i += 32) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(chunk(i / kChunks, i % kChunks)));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w[k]), "r"(zero));
                    }
                    if (__any_sync(0xffffffffu, (sum & 0x7fff7fffu) != 0)) {
                        const int slot = n % kRgUnits;
                        int* const col = bad + slot * D;
                        if (!any_bad)
#pragma unroll 1
                            for (int i = lane; i < D; i += 32) __stcg(col + i, 0x7fffffff);
                        any_bad = true;
                        __threadfence();
                        __syncwarp();
#pragma unroll 1
                        for (int i = r0 * kChunks + lane; i < r1 * kChunks; i += 32) {
                            const uint32_t a = chunk(i / kChunks, i % kChunks);
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                uint16_t e;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(a + 2 * k));
                                if ((e & 0x7f80) != 0x7f80) continue;
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(a + 2 * k), "h"((uint16_t)0) : "memory");
                                atomicMin(col + (i % kChunks) * 8 + k, t1 + i / kChunks);
                            }
                        }
                        __threadfence();
                        __syncwarp();
                        if (lane == 0) *reinterpret_cast<volatile int*>(bad_flag + slot) = 1 + (int)(n / kRgUnits);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(mended + 8 * s);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(u_empty + 8 * (n % kRgUnits));
            }
            // Leave only once all copies have landed.
            if (lane == 0)
#pragma unroll 1
                for (int i = 0; i < 18; ++i)
                    if (issued >> i & 1)
                        rg_wait_longer(i < 16 ? full + 8 * i : q_full + 8 * (i - 16), parity >> i & 1, tmo);
        } else if (elect_one()) {
            // -------------------------------------------------------- products
            // One thread, elected so that the compiler knows of no other: from a branch
            // on the lane every product's operands were made uniform by themselves (the
            // long prompt 1932 us, 1758 with a converged warp that elects for each batch
            // of products, 1545 like this).
            constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
            constexpr uint64_t kDescK = smem_desc_base(16, 1024), kDescV = smem_desc_base(kBlock, 1024);
            struct Now {
                int a, b, all, j0, lim;          // steps of A, B, both
                uint32_t it, dual;               // 0 or 1
            } u = {0, 0, 1, 0, 0, 0, 0}, next = u;   // a unit without steps leads in the first
            uint32_t n = 0, it = 0, phases = 0, mends = 0;
            bool ok = true, issued = false;
            auto wait_one = [&](uint32_t bar, uint32_t parity) {
                ok = ok && wait(bar, parity);
            };
            auto wait_next = [&](uint32_t bar, int bit, uint32_t flip) {
                wait_one(bar, (phases >> bit) ^ flip);
                phases ^= 1u << bit;
            };
            // The next unit. One without key tiles is a step of its own, in which nothing but the
            // unit behind it is taken up: this thread must not look further ahead before it has
            // issued the last product of a unit that the output warps hold.
            auto fetch = [&]() {
                if (!next_unit(n)) return false;
                const RgUnit& f = units[n % kRgUnits];
                if (!f.valid) return false;
                const RgSteps st(f);
                next = {st.a, st.b, max(max(st.a, st.b), 1), f.j0, f.pos0, it, st.dual};
                it += max(f.tiles[0], f.tiles[1]);
                mbar_arrive(u_empty + 8 * (n % kRgUnits));
                ++n;
                return true;
            };
            // S_X for K tile i of all.
            auto scores = [&](uint32_t i, int x, bool first, bool last, bool release) {
                const uint32_t s = i % SK;
                if (first) wait_next(q_full + 8 * x, x, 0);
                if (RS::kApart) wait_next(s_free + 8 * x, 6 + x, 1);
                wait_one(full + 8 * s, i / SK);
                if (!ok) return;
                tc_fence_after();
                const uint64_t a = kDescK + ((q_s + x * kTile) >> 4), b = kDescK + ((ring_s + s * kTile) >> 4);
                const uint32_t to = tmem + RS::kColS + x * 128;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
                    umma_bf16(to, a + off, b + off, kIdescS, k > 0 ? 1u : 0u);
                }
                umma_commit(s_full + 8 * x);
                if (last) umma_commit(q_empty + 8 * x);
                if (release) umma_commit(empty + 8 * s);
                issued = true;
            };
            // O_X += P_X V for V tile i of all.
            auto values = [&](uint32_t i, int x, bool fresh, bool mend, bool first, bool last, bool release) {
                const uint32_t s = SK + i % SV;
                if (fresh) {
                    wait_one((mend ? mended : full) + 8 * s, mend ? mends >> s : i / SV);
                    if (mend) mends ^= 1u << s;
                }
                if (first) wait_next(o_empty + 8 * x, 4 + x, 1);
                const uint64_t b = kDescV + ((ring_s + s * kTile) >> 4);
                const uint32_t to = tmem + RS::kColO + x * D, a = tmem + RS::kColP + x * RS::kStepP;
                wait_one(p_full + 8 * x, phases >> (2 + x));
                if (!ok) return;
                tc_fence_after();
                phases ^= 4u << x;
#pragma unroll
                for (int k = 0; k < kRgTile / 16; ++k)
                    umma_bf16_ts(to, a + (k >> 2) * RS::kHalfP + (k & 3) * 8, b + k * (16 * 128 >> 4), kIdescO,
                                 !first || k > 0 ? 1u : 0u);
                if (RS::kApart) umma_commit(pv_done + 8 * x);
                if (last) umma_commit(o_full + 8 * x);
                if (release) umma_commit(empty + 8 * s);
            };
            bool have = true;
            while (have) {
                bool more = false;
                int j = 0;
                if (!RS::kApart && !u.dual && ok) {
                    // Steps after which both tiles go on in this unit: what one thread spends on
                    // instructions here, the tensor cores wait for.
                    const int steady = min(u.a, u.b) - 1;
                    uint32_t sv = u.it % SV, tv = (u.it / SV) & 1, sk = (u.it + 1) % SK, tk = ((u.it + 1) / SK) & 1;
#pragma unroll 1
                    for (; j < steady && ok; ++j) {
                        const uint32_t v_lo = (ring_s + (SK + sv) * kTile) >> 4, k_lo = (ring_s + sk * kTile) >> 4;
                        const bool mend = (u.j0 + j) * kRgTile + kRgTile - 1 > u.lim;
                        wait_one((mend ? mended : full) + 8 * (SK + sv), mend ? mends >> (SK + sv) : tv);
                        if (mend) mends ^= 1u << (SK + sv);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t to = tmem + RS::kColO + x * D, a = tmem + RS::kColP + x * RS::kStepP;
                            if (j == 0) wait_next(o_empty + 8 * x, 4 + x, 1);
                            wait_one(p_full + 8 * x, phases >> (2 + x));
                            phases ^= 4u << x;
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < kRgTile / 16; ++k)
                                umma_bf16_ts(to, a + (k >> 2) * RS::kHalfP + (k & 3) * 8, kDescV + (v_lo + k * (16 * 128 >> 4)),
                                             kIdescO, j > 0 || k > 0 ? 1u : 0u);
                            if (x == 1) umma_commit(empty + 8 * (SK + sv));
                            if (x == 0) wait_one(full + 8 * sk, tk);
                            if (!ok) break;
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
                                umma_bf16(tmem + RS::kColS + x * 128, kDescK + (((q_s + x * kTile) >> 4) + off), kDescK + (k_lo + off),
                                          kIdescS, k > 0 ? 1u : 0u);
                            }
                            umma_commit(s_full + 8 * x);
                            if (j + 2 == (x ? u.b : u.a)) umma_commit(q_empty + 8 * x);
                            if (x == 1) umma_commit(empty + 8 * sk);
                        }
                        if (++sv == SV) sv = 0, tv ^= 1;
                        if (++sk == SK) sk = 0, tk ^= 1;
                    }
                }
#pragma unroll 1
                for (; j < u.all; ++j) {
                    const bool end = j + 1 == u.all;
                    if (end) more = fetch();
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        const int steps = x ? u.b : u.a;
                        // What S_X holds next: this unit's next tile of X, or the next unit's first.
                        bool go = j + 1 < steps, lead = false;
                        const int v = (j << u.dual) + (x & u.dual);
                        uint32_t i = u.it + v + (1 << u.dual);
                        bool last = j + 2 == steps, release = u.dual || x == 1 || j + 1 >= u.b;
                        if (!go && end && more) {
                            const int to = x ? next.b : next.a;
                            go = lead = to > 0;
                            i = next.it + (x & next.dual);
                            last = to == 1;
                            release = next.dual || x == 1 || next.b == 0;
                        }
                        if (RS::kApart && go) scores(i, x, lead, last, release);
                        if (j < steps)
                            values(u.it + v, x, u.dual || x == 0 || j >= u.a,
                                   (u.j0 + v) * kRgTile + kRgTile - 1 > u.lim, j == 0, j + 1 == steps,
                                   u.dual || x == 1 || j >= u.b);
                        if (!RS::kApart && go) scores(i, x, lead, last, release);
                    }
                }
                u = next;
                have = more;
            }
            // elect_one picks the same thread each time: its commit covers all products.
            if (issued) {
                umma_commit(fin);
                if (!rg_wait_longer(fin, 0, tmo)) atomicOr(p.status, kStatusTimeout);
            }
        }
    } else if (warp >= kRgOut) {
        // ---------------------------------------------------------------- outputs
        const int row = threadIdx.x & 127;
        const int tok = p.by_heads(row);
        const bool in_tile = row < p.tq * p.heads_per_group;
        uint32_t nt = 0;                         // bit x: phases of O_x
        for (uint32_t n = 0; next_unit(n); ++n) {
            __syncwarp();
            const RgUnit& u = units[n % kRgUnits];
            if (!u.valid) break;
            const int slot = u.slot;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (u.tokens[x] == 0) continue;
                const bool some = u.tiles[x] > 0, dual = RgSteps(u).dual;
                float m = -INFINITY, l = 0.f, a0 = 1.f, a1 = 0.f;      // factors of O_A, O_B if both have the rows
                bool ok = true;
                if (some) {
                    const uint64_t whole = kRgTileNs * u.tiles[x];         // these wait for all of the unit
                    ok = !*abort_flag && wait(ml_full + 8 * x, nt >> x, whole) && wait(o_full + 8 * x, nt >> x);
                    nt ^= 1u << x;
                    if (dual) {
                        ok = ok && wait(ml_full + 8, nt >> 1) && wait(o_full + 8, nt >> 1);
                        nt ^= 2u;
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
                const bool valid = in_tile && tok < u.tokens[x];
                if (ok) {
                    tc_fence_after();
                    if (some) {
                        const float2 y = ml[x * 128 + row];
                        m = y.x;
                        l = y.y;
                        if (dual) {
                            const float2 z = ml[128 + row];
                            const float top = fmaxf(m, z.x);
                            a0 = l == 0.f ? 0.f : fast_exp2(m - top);
                            a1 = z.y == 0.f ? 0.f : fast_exp2(z.x - top);
                            l = l * a0 + z.y * a1;
                            m = top;
                        }
                    }
                    const bool flagged = *reinterpret_cast<volatile int*>(bad_flag + n % kRgUnits) == 1 + (int)(n / kRgUnits);
                    // A row that sees a key somewhere has an O wherever its tile has one, of zeros where
                    // it sees none of the keys. Weights that are 0 (far below the row's largest
                    // score) multiply it all the same, so that a NaN in V stays one.
                    const int lim = u.pos0 + x * p.tq + tok;
                    const size_t orow = (size_t)(u.row0 + x * p.tq + tok) * p.H + (size_t)u.g * p.heads_per_group +
                                        (row - tok * p.heads_per_group);
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    float* const part = p.part + (size_t)max(slot, 0) * rg_slot_floats(D);
                    const int r = x * 128 + row;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        const uint32_t o_t = tmem + ((uint32_t)((warp & 3) * 32) << 16) + RS::kColO + c;
                        if (some) {
                            tmem_ld16(o_t + x * D, o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0u;
                        }
                        if (dual) {
                            uint32_t b[16];
                            tmem_ld16(o_t + D, b);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(fmaf(__uint_as_float(b[i]), a1, __uint_as_float(o[i]) * a0));
                        }
                        if (c + 16 == D && some) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(o_empty + 8 * x);
                            if (lane == 0 && dual) mbar_arrive(o_empty + 8);
                        }
                        if (lim < 0)
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0u;
                        if (valid && slot < 0) {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                w[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
                            store32(p.out + orow * D + c, w, p.wide);
                        } else if (valid) {
                            store32(part + (size_t)r * D + c, o, true);
                            store32(part + (size_t)r * D + c + 8, o + 8, true);
                        }
                        __syncwarp();
                    }
                    if (flagged && valid) {                      // a value that is not finite, where the row sees it
#pragma unroll 1
                        for (int c = 0; c < D; ++c) {
                            if (__ldcg(bad + (n % kRgUnits) * D + c) > lim) continue;
                            if (slot < 0)
                                p.out[orow * D + c] = 0x7fc0;
                            else
                                part[(size_t)r * D + c] = __uint_as_float(0x7fc00000u);
                        }
                    }
                    if (valid) {
                        if (slot >= 0) {
                            part[256 * D + r] = m;
                            part[256 * D + 256 + r] = l;
                        } else if (p.lse) {
                            p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                        }
                    }
                }
            }
            if (slot >= 0) {
                // The CTA whose part arrives last merges the unit, once it has no other work:
                // its own part of a unit that goes on in the next CTA is its last one. The
                // barrier orders the part's stores before the arrival, which releases them.
                named_sync(9, 128);
                if (row == 0 && arrive_last(p.counters + u.counter, p.tag, u.parts)) todo[(*todos)++] = u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty + 8 * (n % kRgUnits));
        }
    } else {
        // ---------------------------------------------------------------- softmax
        // Half h of tile X's keys. Nothing here is left out when a wait has expired: the
        // two warps of the same rows meet at named barriers, which have no time limit.
        const int x = warp >> 3, h = (warp >> 2) & 1, row = threadIdx.x & 127;
        const int tok = p.by_heads(row);
        const bool in_tile = row < p.tq * p.heads_per_group;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_t = lanes + RS::kColS + x * 128 + h * 64, p_t = lanes + RS::kColP + x * RS::kStepP + h * RS::kHalfP;
        const uint32_t o_t = lanes + RS::kColO + x * D + h * (D / 2);
        const int pair = 1 + x * 4 + (warp & 3);
        float* const my_top = top_s + (x * 2 + h) * 128 + row;
        const float* const other_top = top_s + (x * 2 + (h ^ 1)) * 128 + row;
        // Scores read at a time. 32 wait half as often, 16 leave room for registers: 8 prompts of
        // 1024, D 64 41.3 us against 43.0; one of 16384, D 128 1432 us against 1422.
        constexpr int kRead = D == 64 ? 32 : 16;
        uint32_t ns = 0, nu = 0;                 // tiles, units so far
        for (uint32_t n = 0; next_unit(n); ++n) {
            __syncwarp();
            const RgUnit& u = units[n % kRgUnits];
            if (!u.valid) break;
            const RgSteps st(u);
            const int tiles = x ? st.b : st.a, xr = st.dual ? 0 : x;
            const int lim = in_tile && tok < u.tokens[xr] ? u.pos0 + xr * p.tq + tok : -1;
            int t0 = (u.j0 + (st.dual ? x : 0)) * kRgTile + h * 64;      // first key of this half
            const int step = st.dual ? 2 * kRgTile : kRgTile;
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty + 8 * (n % kRgUnits));
            if (tiles == 0) continue;
            const bool idle = __all_sync(0xffffffffu, lim < 0);      // no row of this warp sees anything
            const float slack = lim < 0 ? INFINITY : kRgSlack;       // rows without a token hold anything
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++ns, t0 += step) {
                wait(s_full + 8 * x, ns);
                __syncwarp();
                tc_fence_after();
                bool settled = false;            // O_X holds all earlier keys, P is free
                const bool cut = __any_sync(0xffffffffu, (unsigned)lim < t0 + 63u);     // some row sees a part of the keys
                // The reference is the one of the tiles before as long as the weights' sum shows
                // that no score exceeds it by much; otherwise (and with a row's first tile) the
                // tile's maximum is taken first.
                for (bool fresh = j == 0; !idle; fresh = true) {
                    if (fresh) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 64; c += kRead) {
                            uint32_t s[kRead];
                            load_scores(s_t + c, s);
                            if (cut) hide(s, lim - t0 - c);
                            float t[2] = {top, top};
#pragma unroll
                            for (int i = 0; i < kRead; i += 4) {
                                t[0] = fmax3(t[0], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                                t[1] = fmax3(t[1], __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
                            }
                            top = fmaxf(t[0], t[1]);
                        }
                        *my_top = top;
                        named_sync(pair, 64);
                        top = fmaxf(top, *other_top) * p.scale_log2;
                        const float mn = fmaxf(top, m);
                        if (j > 0) {
                            if (RS::kApart && !settled) {
                                wait(pv_done + 8 * x, ns - 1);
                                __syncwarp();
                                tc_fence_after();
                                settled = true;
                            }
                            const float a = mn > m ? fast_exp2(m - mn) : 1.f;
#pragma unroll 1
                            for (int c = 0; c < D / 2; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(o_t + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                                tmem_st16(o_t + c, o);
                            }
                            l *= a;
                        }
                        m = mn;
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float2 scale = make_float2(p.scale_log2, p.scale_log2), neg = make_float2(-ref, -ref);
                    float2 sum[2] = {};
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 64; c += kRead) {
                        uint32_t s[kRead];
                        load_scores(s_t + c, s);
                        if (cut) hide(s, lim - t0 - c);
                        weigh(s, scale, neg, sum, w + c / 2);
                    }
                    sum[0] = add_x2(sum[0], sum[1]);
                    const float all = sum[0].x + sum[0].y;
                    if (!fresh && pair_any(pair, all > slack || (m == -INFINITY && t0 <= lim))) continue;
                    if (RS::kApart) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + 8 * x);
                        if (ns > 0 && !settled) wait(pv_done + 8 * x, ns - 1);
                        __syncwarp();
                        tc_fence_after();
                    }
                    tmem_st32(p_t, w);
                    l += all;
                    tmem_st_wait();
                    break;
                }
                if (RS::kApart && idle) {
                    // No arrival for this tile's P may count for the one before.
                    if (lane == 0) mbar_arrive(s_free + 8 * x);
                    if (ns > 0) wait(pv_done + 8 * x, ns - 1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * x);
            }
            if (!idle) {
                if (h) sum_s[x * 128 + row] = l;
                named_sync(pair, 64);
                if (!h) l += sum_s[x * 128 + row];
            }
            if (!h) {
                // The unit before has been read from here once its O is given back.
                wait(o_empty + 8 * x, nu ^ 1);
                ml[x * 128 + row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full + 8 * x);
            }
            ++nu;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kRgMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // All copies have landed and all products are done: Q's and the ring's room is free.
    uint32_t phases = 0;
#pragma unroll 1
    for (int i = 0; i < *todos; ++i)
        rg_merge<D>(p, todo[i], smem_raw, (2 + S) * kTile, merge_bar, phases);
}

template <int D, bool PAGED>
cudaError_t launch_ragged(const RaggedLaunch& a) {
    using RS = RgShape<D>;
    // The shared-memory opt-in is per function and per device.
    static std::atomic<unsigned long long> attr_set_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(attr_set_mask.load() & bit)) {
        e = cudaFuncSetAttribute(gqa_ragged_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 RS::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set_mask.fetch_or(bit);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(kRgThreads);
    cfg.dynamicSmemBytes = RS::kSmemBytes;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gqa_ragged_kernel<D, PAGED>, a.tm_q, a.tm_k, a.tm_v, a.p);
}

}  // namespace gqa
