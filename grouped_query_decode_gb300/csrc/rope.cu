// Rotary positions (gqa_rope) and the append of new tokens to bf16 pages
// (gqa_append_paged), which rotates keys and queries on the way.
//
// Pair i of a head, (a, b), at position t becomes
//     a' = gain (a cos(t f_i) - b sin(t f_i)),   b' = gain (b cos(t f_i) + a sin(t f_i)).
// The angle is kept as a fraction of a turn in 64-bit fixed point: f_i / 2 pi is
// an integer multiple of 2^-64 turns, whose product with t modulo 2^64 is exact
// for every 32-bit t, so no position loses accuracy (a product in fp32 is off by
// 0.03 radians at t = 2^20). Sine and cosine are fp32, computed once per token
// and pair and shared by all heads through shared memory; the products are fp32
// and rounded once, to bf16.
//
// What bounds it: bytes, every row read and written once; 64 tokens take the launch
// and one token's chain of dependent reads (2.6 us in a graph, the append 3.6).
// Measured on one GB300 (copy 6.79 TB/s), 32/8 heads, D 128: 16384 tokens with half
// of each head rotated 53.9 us, 6.2 TB/s; 5818 tokens of six sequences appended to
// 64-token pages 27 us, 5.3 TB/s (23000 of 24: 91 us, 6.6 TB/s).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gqa_decode.h"
#include "gqa_device.cuh"
#include "gqa_launch.h"
#include "gqa_paged_fp8.h"
#include "gqa_rope_step.h"

namespace gqa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;           // tokens of a CTA, a warp each for angles and addresses
constexpr int kMostPairs = 64;

struct RopeParams {
    unsigned long long step[kMostPairs]; // f_i as 2^-64 turns per position
    float gain, sign;                    // sign -1: the transpose
    int half, interleaved;               // pairs; 0 pairs: no rotation
    const uint16_t *q, *k, *v;           // v: append only
    uint16_t *q_out, *k_out, *v_out;     // append: k_out, v_out are the pages
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    const int32_t* positions;            // rope only
    const int32_t *cu, *lens, *table;    // append only
    int N, B, H, G, page_shift, num_pages, max_pages;
    int tokens;                          // of a CTA
    FastDiv by_rows;                     // by the rows (heads) of a token
};

// Sequence of token n: the last b with cu[b] <= n (cu ascending), or -1 where n is
// behind the last sequence. The warp narrows by 32 at a step.
__device__ int find_sequence(const int32_t* cu, int B, int n, int lane) {
    int lo = 0, count = B + 1;           // the answer is in [lo, lo + count), cu[lo] <= n
    while (count > 1) {
        const int step = (count + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < count && __ldg(cu + at) <= n;
        const unsigned votes = __ballot_sync(0xffffffffu, below);
        const int last = votes ? 31 - __clz(votes) : 0;
        const int end = lo + count;
        lo += last * step;
        count = min(step, end - lo);
    }
    return lo;
}

// The append's rows come from three tensors and go through a table: eight CTAs on an SM
// (32 registers) have more of them under way (24 chunks 95.6 us, 91.1 so); the rotation
// alone loses by it (16384 tokens 54.1 us, 54.6).
template <int D, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, APPEND ? 8 : 6) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float cos_s[kRopeTokens][kMostPairs];
    __shared__ __align__(16) float sin_s[kRopeTokens][kMostPairs];
    __shared__ long long page_at[kRopeTokens];     // element of the token's row of KV head 0, -1: not written
    __shared__ bool used[kRopeTokens];
    __shared__ __align__(16) uint16_t row_s[kRopeThreads / 32][D];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * p.tokens;
    pdl_launch_dependents();
    pdl_wait_primary();
    if (warp < p.tokens) {
        const int n = n0 + warp;
        bool use = n < p.N;
        int t = 0;
        if (use && !APPEND) t = __ldg(p.positions + n);
        if (use && APPEND) {
            const int b = find_sequence(p.cu, p.B, n, lane);
            use = b < p.B && __ldg(p.cu + b) <= n;
            if (use) {
                const int first = max(0, min(__ldg(p.cu + b), p.N));
                const int end = max(first, min(__ldg(p.cu + b + 1), p.N));
                const long long most = (long long)p.max_pages << p.page_shift;
                t = (int)min((long long)max(__ldg(p.lens + b), 0), most) - end + n;
                if (lane == 0) {
                    long long at = -1;
                    if (t >= 0) {
                        const int page = __ldg(p.table + (size_t)b * p.max_pages + (t >> p.page_shift));
                        if ((unsigned)page < (unsigned)p.num_pages)
                            at = ((((long long)page * p.G) << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * D;
                    }
                    page_at[warp] = at;
                }
            }
        }
        if (lane == 0) used[warp] = use;
        if (use)
            for (int i = lane; i < p.half; i += 32) {
                const unsigned long long turn = (unsigned long long)(long long)t * p.step[i];
                float s, c;
                sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
                cos_s[warp][i] = c * p.gain;
                sin_s[warp][i] = s * p.gain * p.sign;
            }
    }
    __syncthreads();

    const int rows = p.H + p.G * (APPEND ? 2 : 1);
    const int total = min(p.tokens, p.N - n0) * rows;
    // Row r of a token: its queries, then keys, then values. Returns false for a row that stays out.
    auto where = [&](int item, int& w, bool& turned, const uint16_t*& from, uint16_t*& to) {
        w = p.by_rows(item);
        int r = item - w * rows;
        const int n = n0 + w;
        if (!used[w]) return false;
        turned = p.half > 0;
        if (r < p.H) {
            from = p.q + (size_t)n * p.q_stride + r * D;
            to = p.q_out + (size_t)n * p.q_out_stride + r * D;
            return true;
        }
        r -= p.H;
        const bool value = APPEND && r >= p.G;
        if (value) {
            r -= p.G;
            turned = false;
        }
        from = (value ? p.v + (size_t)n * p.v_stride : p.k + (size_t)n * p.k_stride) + r * D;
        if (APPEND) {
            if (page_at[w] < 0) return false;
            to = (value ? p.v_out : p.k_out) + page_at[w] + (((long long)r * D) << p.page_shift);
        } else {
            to = p.k_out + (size_t)n * p.k_out_stride + r * D;
        }
        return true;
    };

    if (!p.interleaved && (p.half & 7)) {
        // Halves that do not start on 16 bytes: a warp per row, through shared memory. Half of
        // the lanes copy, one row is under way, and pairs are read and written 2 bytes at a
        // time: 16384 tokens, 32/8 heads, D 128, 50 elements rotated take 99 us, 48 take 53;
        // 5818 tokens appended 42 us for 27.
        uint16_t* mine = row_s[warp];
        for (int item = warp; item < total; item += kRopeThreads / 32) {
            int w;
            bool turned;
            const uint16_t* from;
            uint16_t* to;
            if (!where(item, w, turned, from, to)) continue;
            if (lane < D / 8) *reinterpret_cast<uint4*>(mine + lane * 8) = *reinterpret_cast<const uint4*>(from + lane * 8);
            __syncwarp();
            if (turned)
                for (int i = lane; i < p.half; i += 32) {
                    const float a = __uint_as_float((uint32_t)mine[i] << 16);
                    const float b = __uint_as_float((uint32_t)mine[i + p.half] << 16);
                    const float c = cos_s[w][i], s = sin_s[w][i];
                    const uint32_t y = pack_bf16x2(a * c - b * s, b * c + a * s);
                    mine[i] = (uint16_t)y;
                    mine[i + p.half] = (uint16_t)(y >> 16);
                }
            __syncwarp();
            if (lane < D / 8) *reinterpret_cast<uint4*>(to + lane * 8) = *reinterpret_cast<const uint4*>(mine + lane * 8);
            __syncwarp();
        }
        return;
    }

    // A thread takes two 16-byte chunks of a row: the same chunk of both halves, or
    // two neighbouring ones (neighbouring pairs, and what is not rotated).
    constexpr int kItems = D / 16;
    const int i = threadIdx.x % kItems;
    for (int item = threadIdx.x / kItems; item < total; item += kRopeThreads / kItems) {
        int w;
        bool turned;
        const uint16_t* from;
        uint16_t* to;
        if (!where(item, w, turned, from, to)) continue;
        const bool halves = !p.interleaved && i * 8 < p.half;
        const int c0 = halves ? i * 8 : i * 16, c1 = halves ? c0 + p.half : c0 + 8;
        // Past the halves, the chunks of [2 half, D) in order: 16 i is at or past 2 half there.
        uint4 x = *reinterpret_cast<const uint4*>(from + c0), y = *reinterpret_cast<const uint4*>(from + c1);
        uint32_t* const a = reinterpret_cast<uint32_t*>(&x);
        uint32_t* const b = reinterpret_cast<uint32_t*>(&y);
        if (turned && halves) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 c = *reinterpret_cast<const float2*>(&cos_s[w][c0 + 2 * k]);
                const float2 s = *reinterpret_cast<const float2*>(&sin_s[w][c0 + 2 * k]);
                const float a0 = __uint_as_float(a[k] << 16), a1 = __uint_as_float(a[k] & 0xffff0000u);
                const float b0 = __uint_as_float(b[k] << 16), b1 = __uint_as_float(b[k] & 0xffff0000u);
                a[k] = pack_bf16x2(a0 * c.x - b0 * s.x, a1 * c.y - b1 * s.y);
                b[k] = pack_bf16x2(b0 * c.x + a0 * s.x, b1 * c.y + a1 * s.y);
            }
        } else if (turned && p.interleaved) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int pair = i * 8 + k;
                if (pair >= p.half) break;
                uint32_t& z = k < 4 ? a[k & 3] : b[k & 3];
                const float c = cos_s[w][pair], s = sin_s[w][pair];
                const float z0 = __uint_as_float(z << 16), z1 = __uint_as_float(z & 0xffff0000u);
                z = pack_bf16x2(z0 * c - z1 * s, z1 * c + z0 * s);
            }
        }
        *reinterpret_cast<uint4*>(to + c0) = x;
        *reinterpret_cast<uint4*>(to + c1) = y;
    }
}

template <int D, bool APPEND>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.N + p.tokens - 1) / p.tokens);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<D, APPEND>, p);
}

int check_rope(const gqa_rope_t* r, int D) {
    if (r->dims < 2 || r->dims > D || (r->dims & 1)) return GQA_ERR_INVALID_ARG;
    if (!std::isfinite(r->gain) || std::fabs(r->gain) > 3e38) return GQA_ERR_INVALID_ARG;
    for (int i = 0; i < r->dims / 2; ++i)
        if (!std::isfinite(r->inv_freq[i]) || std::fabs(r->inv_freq[i]) > 1e15) return GQA_ERR_INVALID_ARG;
    return GQA_OK;
}

void set_rope(RopeParams* p, const gqa_rope_t* r, bool inverse) {
    p->half = r ? r->dims / 2 : 0;
    p->interleaved = r ? r->interleaved != 0 : 0;
    p->gain = r ? (float)r->gain : 1.f;
    p->sign = inverse ? -1.f : 1.f;
    for (int i = 0; i < p->half; ++i) p->step[i] = rope_step(r->inv_freq[i]);
}

bool aligned(const void* x, unsigned mask) { return (reinterpret_cast<uintptr_t>(x) & mask) == 0; }

// A packed tensor [N, heads, D] whose tokens are `stride` elements apart.
int check_rows(const void* x, long long stride, int heads, int D) {
    if (stride < (long long)heads * D) return GQA_ERR_INVALID_ARG;
    return aligned(x, 15u) && (stride & 7) == 0 ? GQA_OK : GQA_ERR_MISALIGNED;
}

// A tensor and what it is rotated into: apart, or the same with the same stride.
int check_pair(const void* x, long long stride, const void* out, long long out_stride, int N, int heads, int D) {
    int st = check_rows(x, stride, heads, D);
    if (st == GQA_OK) st = check_rows(out, out_stride, heads, D);
    return st != GQA_OK || x != out || stride == out_stride || N == 1 ? st : GQA_ERR_INVALID_ARG;
}

// Tokens of a CTA: one while there are few (a token's rows are then spread over all of
// its threads), two from sixteen CTAs per SM, `most` where that still makes sixteen. 16384
// tokens rotated, 32/8 heads, D 128: 53.8 us with four, 55.8 with two, 57.2 with eight; 8192
// 30.4 with four, 30.0 with two. 24 chunks appended: D 64 50.1 us with four, 51.6 with two;
// D 128 94.8 with four, 91.1 with two.
int tokens_per_cta(int N, int sms, int most) { return N >= sms * 16 * kRopeTokens ? most : N >= sms * 16 ? 2 : 1; }

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_rope_init(gqa_rope_t* rope, int D, int dims, int interleaved, double base, int scaling, double factor,
                  double original, double low, double high) {
    if (!rope || D <= 0 || dims < 2 || dims > D || (dims & 1)) return GQA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (!(base > 1.0) || !std::isfinite(base)) return GQA_ERR_INVALID_ARG;
    if (scaling < GQA_ROPE_PLAIN || scaling > GQA_ROPE_YARN) return GQA_ERR_INVALID_ARG;
    if (scaling != GQA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return GQA_ERR_INVALID_ARG;
    if (scaling >= GQA_ROPE_BANDS && (!(original > 0.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) ||
                                      !std::isfinite(high)))
        return GQA_ERR_INVALID_ARG;
    constexpr double kTurn = 6.283185307179586477;
    rope->dims = dims;
    rope->interleaved = interleaved != 0;
    rope->gain = 1.0;
    for (double& f : rope->inv_freq) f = 0.0;
    if (scaling == GQA_ROPE_BASE && dims > 2) base *= std::pow(factor, (double)dims / (dims - 2));
    // The pair that makes `turns` turns over the original context.
    auto pair_of = [&](double turns) { return dims * std::log(original / (turns * kTurn)) / (2 * std::log(base)); };
    double first = 0, last = 0;
    if (scaling == GQA_ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), (double)(dims - 1));
        rope->gain = 1.0 + 0.1 * std::log(factor);
    }
    for (int i = 0; i < dims / 2; ++i) {
        double f = std::pow(base, -2.0 * i / dims);
        double slow = 0.0;               // share of the pair that the factor slows
        if (scaling == GQA_ROPE_LINEAR) slow = 1.0;
        if (scaling == GQA_ROPE_BANDS) slow = 1.0 - (original * f / kTurn - low) / (high - low);
        if (scaling == GQA_ROPE_YARN) slow = (i - first) / std::fmax(last - first, 0.001);
        slow = std::fmin(std::fmax(slow, 0.0), 1.0);
        if (slow > 0.0) f = f * (1.0 - slow) + f / factor * slow;
        rope->inv_freq[i] = f;
    }
    return GQA_OK;
}

int gqa_rope(const gqa_rope_t* rope, const void* q, const void* k, const int32_t* positions, void* q_out,
             void* k_out, int N, int H, int G, int D, long long q_stride, long long k_stride,
             long long q_out_stride, long long k_out_stride, int inverse, cudaStream_t stream) {
    if (N == 0 && rope && H >= 0 && G >= 0 && D > 0) return GQA_OK;      // tensors without rows have no address
    if (!rope || !positions || (!q && !k) || (q && !q_out) || (k && !k_out)) return GQA_ERR_INVALID_ARG;
    if (N < 0 || (q && H <= 0) || (k && G <= 0) || D <= 0) return GQA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    int st = check_rope(rope, D);
    if (st != GQA_OK) return st;
    if (!q) H = 0;
    if (!k) G = 0;
    if ((long long)N * H + (long long)N * G >= (1ll << 31) || (long long)H + G >= (1 << 20)) return GQA_ERR_UNSUPPORTED;
    if (!aligned(positions, 3u)) return GQA_ERR_MISALIGNED;
    if (q && (st = check_pair(q, q_stride, q_out, q_out_stride, N, H, D)) != GQA_OK) return st;
    if (k && (st = check_pair(k, k_stride, k_out, k_out_stride, N, G, D)) != GQA_OK) return st;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    RopeParams p = {};
    set_rope(&p, rope, inverse != 0);
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(k_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.positions = positions;
    p.N = N;
    p.H = H;
    p.G = G;
    p.tokens = tokens_per_cta(N, sms, kRopeTokens);
    p.by_rows = FastDiv((unsigned)(H + G));
    const cudaError_t e = D == 64 ? launch_rope<64, false>(p, stream) : launch_rope<128, false>(p, stream);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

int gqa_append_paged(const gqa_rope_t* rope, const void* q, const void* k_new, const void* v_new, void* q_out,
                     void* k_pages, void* v_pages, const int32_t* block_table, const int32_t* cu_new,
                     const int32_t* seq_lens, int N, int B, int H, int G, int D, long long q_stride,
                     long long k_stride, long long v_stride, long long q_out_stride, int page_size, int num_pages,
                     int max_pages_per_seq, cudaStream_t stream) {
    if (N == 0 && B > 0 && G > 0 && D > 0) return GQA_OK;
    if (!k_new || !v_new || !k_pages || !v_pages || !block_table || !cu_new || !seq_lens || (q && !q_out))
        return GQA_ERR_INVALID_ARG;
    if (N < 0 || B <= 0 || (q && H <= 0) || G <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0 || max_pages_per_seq <= 0)
        return GQA_ERR_INVALID_ARG;
    if (q && H % G != 0) return GQA_ERR_HEAD_RATIO;
    if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1))) return GQA_ERR_UNSUPPORTED;
    int st = rope ? check_rope(rope, D) : GQA_OK;
    if (st != GQA_OK) return st;
    if (!q) H = 0;
    if ((long long)max_pages_per_seq * page_size >= (1ll << 31) - 128 || (long long)num_pages * G >= (1ll << 31) ||
        (long long)N * (H + 2ll * G) >= (1ll << 31) || H + 2ll * G >= (1 << 20) ||
        B >= (1ll << 31) - 33)                           // find_sequence counts B + 1 and 31 more
        return GQA_ERR_UNSUPPORTED;
    if (!aligned(block_table, 3u) || !aligned(cu_new, 3u) || !aligned(seq_lens, 3u) || !aligned(k_pages, 15u) ||
        !aligned(v_pages, 15u))
        return GQA_ERR_MISALIGNED;
    if (q && (st = check_pair(q, q_stride, q_out, q_out_stride, N, H, D)) != GQA_OK) return st;
    if ((st = check_rows(k_new, k_stride, G, D)) != GQA_OK || (st = check_rows(v_new, v_stride, G, D)) != GQA_OK)
        return st;
    int sms;
    unsigned* status;
    st = current_device(&sms, &status);
    if (st != GQA_OK) return st;
    RopeParams p = {};
    set_rope(&p, rope, false);
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_new);
    p.v = static_cast<const uint16_t*>(v_new);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_out = static_cast<uint16_t*>(k_pages);
    p.v_out = static_cast<uint16_t*>(v_pages);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.cu = cu_new;
    p.lens = seq_lens;
    p.table = block_table;
    p.N = N;
    p.B = B;
    p.H = H;
    p.G = G;
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.num_pages = num_pages;
    p.max_pages = max_pages_per_seq;
    p.tokens = tokens_per_cta(N, sms, D == 64 ? kRopeTokens : 2);
    p.by_rows = FastDiv((unsigned)(H + 2 * G));
    const cudaError_t e = D == 64 ? launch_rope<64, true>(p, stream) : launch_rope<128, true>(p, stream);
    return e == cudaSuccess ? GQA_OK : remember_cuda_error(e);
}

}  // extern "C"
