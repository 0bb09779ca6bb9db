// A pair's turns per position (gqa_rope_step.h), compiled for the host. Compiled and
// called by test_rope_step_cpu.py.
#include "gqa_rope_step.h"

extern "C" unsigned long long rope_step(double inv_freq) { return gqa::rope_step(inv_freq); }
