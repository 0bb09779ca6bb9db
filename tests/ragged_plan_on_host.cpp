// How the attention of a packed batch is shared out (gqa_ragged_plan.cuh), compiled
// for the host: every part of every unit that every CTA takes. Compiled and called
// by test_ragged_plan_cpu.py.
#include <cstring>

#include "gqa_ragged_plan.cuh"

using namespace gqa;

extern "C" long long ragged_parts(const int* start, const int* n, const int* T, int B, int tq, int G, int D, int grid,
                                  int* out, long long most) {
    const RgLine line = RgLine::of(tq, G, D);
    long long total = 0, count = 0;
    for (int b = 0; b < B; ++b) total += line.head({start[b], n[b], T[b]}) * G;
    const RgShares sh = RgShares::of(total, grid);
    for (int c = 0; c < sh.ctas; ++c) {
        long long at = 0;
        for (int b = 0; b < B; ++b) {
            const RgSeq s = {start[b], n[b], T[b]};
            const long long head = line.head(s);
            for (int g = 0; g < G; ++g)
                for (int pr = 0; pr < line.pairs(s.n); ++pr) {
                    const long long unit = at + g * head + line.start(s, pr);
                    if (unit >= sh.at(c + 1) || unit + line.length(s, pr) <= sh.at(c)) continue;
                    // where the kernel starts to walk
                    if (unit <= sh.at(c) && line.pair_at(s, sh.at(c) - at - g * head) != pr) return -1;
                    RgUnit u;
                    u.seq = b;
                    u.g = g;
                    if (!rg_unit(line, sh, c, s, pr, unit, &u)) continue;
                    if (count == most) return -2;
                    out[17 * count] = c;
                    std::memcpy(out + 17 * count + 1, &u, 64);
                    ++count;
                }
            at += head * G;
        }
    }
    return count;
}

extern "C" int ragged_ctas(long long total, int grid) { return RgShares::of(total, grid).ctas; }
