// A pair's turns per position, in 64-bit fixed point (host code).
#pragma once

#include <cmath>

namespace gqa {

// inv_freq / 2 pi modulo a turn, in units of 2^-64 turns. The magnitude is converted
// and the sign applied to the result: minus a small frequency lies just below a whole
// turn, where a double is off by up to 2^-54 of it, 7e-7 radians after 2^31 positions.
inline unsigned long long rope_step(double inv_freq) {
    // The product with 1 / 2 pi and what it lacks.
    constexpr double kInv = 0.15915494309189535, kInvRest = -9.839338337591243e-18;
    const double f = std::fabs(inv_freq), turns = f * kInv;
    const double rest = std::fma(f, kInv, -turns) + f * kInvRest;    // below 2^-5
    const unsigned long long step = (unsigned long long)std::ldexp(turns - std::floor(turns), 64) +
                                    (unsigned long long)(long long)std::ldexp(rest, 64);
    return inv_freq < 0 ? 0 - step : step;
}

}  // namespace gqa
