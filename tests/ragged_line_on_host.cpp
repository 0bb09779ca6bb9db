// The numbers that the plan of a packed batch is made of (gqa_ragged_plan.cuh),
// compiled for the host together with ragged_plan_on_host.cpp. Called by
// test_ragged_line_cpu.py.
#include "ragged_plan_on_host.cpp"

// Of unit pr of a sequence: its place from the KV head's start, its length, both in
// keys; least tiles of a part, least keys of a share.
extern "C" void ragged_line(int n, int T, int tq, int G, int D, int pr, long long* out) {
    const RgLine line = RgLine::of(tq, G, D);
    const RgSeq s = {0, n, T};
    out[0] = line.start(s, pr);
    out[1] = line.length(s, pr);
    out[2] = line.head(s);
    out[3] = kRgMinPart;
    out[4] = kRgMinShare;
    out[5] = line.eighths;
    out[6] = line.pad;
}
