// The plan of the paged 8-bit attention (gqa_paged_plan.cuh) compiled for the
// host: the threads of a CTA are fibers that take turns, each running to its
// next exchange with the others. Compiled and called by test_paged_plan_cpu.py.
#include <ucontext.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <vector>

#include <cuda.h>
#include <cuda_runtime_api.h>

#ifndef __noinline__
#define __noinline__
#endif

namespace {

struct Dim {
    unsigned x;
} threadIdx, blockIdx, gridDim;

struct Fiber {
    ucontext_t at;
    std::vector<char> stack;
    int turn = 0;
    bool done = false;
};
std::vector<Fiber> fibers;
ucontext_t scheduler;
uint64_t value_of[2][1024];
int kind_of[2][1024];
bool mixed;                       // threads met in different exchanges

// Deposits a value; when it returns, every thread has deposited its own.
template <class T>
const uint64_t* exchange(int kind, T v) {
    const unsigned t = threadIdx.x;
    Fiber& f = fibers[t];
    const int half = f.turn++ & 1;
    value_of[half][t] = 0;
    std::memcpy(&value_of[half][t], &v, sizeof v);
    kind_of[half][t] = kind;
    swapcontext(&f.at, &scheduler);
    for (size_t i = 0; i < fibers.size(); ++i) mixed |= kind_of[half][i] != kind;
    return value_of[half] + (t & ~31u);
}
template <class T>
T as(uint64_t x) {
    T v;
    std::memcpy(&v, &x, sizeof v);
    return v;
}
template <class T>
T __shfl_sync(unsigned, T v, int src) {
    return as<T>(exchange(1, v)[src & 31]);
}
template <class T>
T __shfl_up_sync(unsigned, T v, int by) {
    const uint64_t* all = exchange(2, v);
    const int lane = threadIdx.x & 31;
    return lane >= by ? as<T>(all[lane - by]) : v;
}
template <class T, class F>
T reduce(int kind, T v, F f) {
    const uint64_t* all = exchange(kind, v);
    T r = as<T>(all[0]);
    for (int i = 1; i < 32; ++i) r = f(r, as<T>(all[i]));
    return r;
}
unsigned __reduce_add_sync(unsigned, unsigned v) {
    return reduce(3, v, [](unsigned a, unsigned b) { return a + b; });
}
unsigned __reduce_min_sync(unsigned, unsigned v) {
    return reduce(4, v, [](unsigned a, unsigned b) { return std::min(a, b); });
}
unsigned __reduce_max_sync(unsigned, unsigned v) {
    return reduce(5, v, [](unsigned a, unsigned b) { return std::max(a, b); });
}
unsigned __ballot_sync(unsigned, bool v) {
    const uint64_t* all = exchange(6, (unsigned)v);
    unsigned m = 0;
    for (int i = 0; i < 32; ++i) m |= (unsigned)(all[i] & 1) << i;
    return m;
}
void __syncwarp() { exchange(7, 0); }
void __syncthreads() { exchange(8, 0); }
int __ffs(unsigned x) { return __builtin_ffs((int)x); }
using std::max;
using std::min;

}  // namespace

#include "gqa_paged_plan.cuh"

namespace {

using namespace gqa;

struct Job {
    const PagedFp8Params* p;
    int rows;
    int* copy;
    P8Plan* plan;                // of each thread
    P8Plan shared;
    long long warp_sum[64];
};
Job* job;
constexpr int kThreads = 64;     // of the plan that all threads make

template <int RP>
void make_plan() {
    const PagedFp8Params& p = *job->p;
    const P8Lens<RP> lens = {p, job->copy};
    if (p.small_plan) {
        job->plan[threadIdx.x] = p8_small_plan<RP>(lens);
    } else {
        p8_make_plan<RP, kThreads>(p, job->copy, &job->shared, job->warp_sum);
        __syncthreads();
        job->plan[threadIdx.x] = job->shared;
    }
}
void fiber_main(int t) {
    threadIdx.x = (unsigned)t;
    if (job->rows == 8) make_plan<8>();
    else if (job->rows == 16) make_plan<16>();
    else make_plan<32>();
    fibers[t].done = true;
}
void run_cta(int threads) {
    fibers.resize(threads);
    for (int t = 0; t < threads; ++t) {
        Fiber& f = fibers[t];
        f.turn = 0;
        f.done = false;
        if (f.stack.empty()) f.stack.resize(64 << 10);
        getcontext(&f.at);
        f.at.uc_stack.ss_sp = f.stack.data();
        f.at.uc_stack.ss_size = f.stack.size();
        f.at.uc_link = &scheduler;
        makecontext(&f.at, reinterpret_cast<void (*)()>(fiber_main), 1, t);
    }
    for (bool left = true; left;) {
        left = false;
        int ended = 0;
        for (int t = 0; t < threads; ++t) {
            if (!fibers[t].done) {
                threadIdx.x = (unsigned)t;
                swapcontext(&scheduler, &fibers[t].at);
            }
            ended += fibers[t].done;
        }
        left = ended < threads;
        mixed |= ended > 0 && left;
    }
}

template <int RP>
int walk(const PagedFp8Params& p, int* copy, const P8Plan& plan, int cta, long long* out, int rows, int cap) {
    const P8Lens<RP> lens = {p, copy};
    P8Walk<RP> w = {plan.left, plan.entry, plan.g, plan.off};
    P8Segment s;
    while (w.next(lens, s)) {
        if (rows == cap) return -2;
        int c0 = cta, n = 1;
        if (s.i0 > 0 || s.i1 < s.n) plan.sharers(s, c0, n);
        const long long row[8] = {cta, s.entry, s.g, s.i0, s.i1, s.n, c0, n};
        std::copy(row, row + 8, out + 8 * (long long)rows++);
    }
    return rows;
}

}  // namespace

extern "C" {

// The segments of all CTAs of a call, eight numbers each: CTA, entry, KV head,
// tiles [i0, i1) of n, the first of the unit's CTAs and their number. Returns
// how many, -1 if threads disagree on the plan, -2 if there are more than `cap`.
int plan_case(int B, int sq, int H, int G, int page_size, int max_pages, const int* lens, int sms, int any_size,
              long long* out, int cap, int* grid) {
    PagedFp8Params p;            // the plan reads what is set here
    p.lens = lens;
    p.B = B;
    p.sq = sq;
    p.H = H;
    p.G = G;
    p.heads_per_group = H / G;
    p.R = H / G * sq;
    const int rows = p8_rows(p.R);
    p.row_tiles = (p.R + rows - 1) / rows;
    p.by_heads = FastDiv((unsigned)p.heads_per_group);
    p.by_row_tiles = FastDiv((unsigned)p.row_tiles);
    p.page_shift = __builtin_ctz((unsigned)page_size);
    p.max_pages = max_pages;
    *grid = p8_grid(B, G, p.R, page_size, max_pages, sms);
    p.small_plan = !any_size && p8_small(B, G, p.R, page_size, max_pages, *grid);
    gridDim.x = (unsigned)*grid;
    int n = 0;
    mixed = false;
    for (int c = 0; c < *grid && n >= 0; ++c) {
        blockIdx.x = (unsigned)c;
        std::vector<int> copy(kP8LenCopy + 4, 0x7e7e7e7e);         // shared memory holds anything
        if (p.small_plan) {                                        // as the kernel does before it plans
            const P8Lens<8> l = {p, copy.data()};
            for (int b = 0; b < 128; ++b) copy[b] = b < B ? l.global(b) : 0;
            copy[kP8LenCopy + 1] = 0;
        }
        const int threads = p.small_plan ? 32 : kThreads;
        std::vector<P8Plan> plan(threads);
        Job j = {};
        j.p = &p;
        j.rows = rows;
        j.copy = copy.data();
        j.plan = plan.data();
        job = &j;
        run_cta(threads);
        for (int t = 1; t < threads; ++t)
            mixed |= plan[t].left != plan[0].left || plan[t].entry != plan[0].entry || plan[t].g != plan[0].g ||
                     plan[t].off != plan[0].off || plan[t].ctas != plan[0].ctas || plan[t].begin != plan[0].begin ||
                     plan[t].end != plan[0].end || plan[t].total != plan[0].total;
        if (mixed) return -1;
        n = rows == 8    ? walk<8>(p, copy.data(), plan[0], c, out, n, cap)
            : rows == 16 ? walk<16>(p, copy.data(), plan[0], c, out, n, cap)
                         : walk<32>(p, copy.data(), plan[0], c, out, n, cap);
    }
    return n;
}

int plan_owner(long long total, int ctas, long long t) {
    P8Plan plan = {};
    plan.total = total;
    plan.ctas = ctas;
    return plan.owner(t);
}

}  // extern "C"
