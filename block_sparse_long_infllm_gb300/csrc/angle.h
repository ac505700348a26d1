// angle.h -- cosine and sine of a fraction of a turn, for the device and, in the tests, the host.
#pragma once

#include <math.h>

#include "places.h"

namespace infllmv2 {

// (cos, sin) of `turn` (in units of 2^-64 of a full one) times scale.
//
// The nearest quarter turn is taken off in integers, so what is left is at most an eighth of a turn and
// small near every zero of either function; a fp32 fraction of the whole turn would be off by up to
// pi 2^-25 (fp32 rows were then off by 5.6e-8 of their norm, now by 3.8e-8).  The rest is the integer n in
// units of 2^-33 of a turn (its rounding: 2 pi 2^-34 < 2^-31), and the angle a + b = 2 pi 2^-33 n two fp32
// numbers.  Taylor's series in z = a^2 up to a^9 and a^10: the first term left out is below 2^-28 of sin
// and 2^-33.  Both end in one product and sum with `scale`: with cos - 1 rounded before it (it is at most
// 0.293: 2^-26), off by half a unit in the last place and 2^-25.4 of the scale.
INFLLMV2_HD void cos_sin_of_turn(unsigned long long turn, float scale, float* c_out, float* s_out) {
    const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
    const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(quarter) << 62));
    const int n = static_cast<int>((rest + (1ll << 30)) >> 31);
    const float two_pi = 6.28318530717958648f * 0x1p-33f, two_pi_low = -1.74845560e-7f * 0x1p-33f;  // their sum is 2 pi 2^-33
    const float nh = static_cast<float>(n), nl = static_cast<float>(n - static_cast<int>(nh));
    const float a = nh * two_pi;
    const float b = fmaf(nl, two_pi, fmaf(nh, two_pi_low, fmaf(nh, two_pi, -a)));
    const float z = a * a, z_low = fmaf(a, a, -z);
    const float s5 = fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    const float c6 = fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
    const float s_rest = fmaf(a * z, s5, fmaf(-0.5f * z, b, b));                            // sin - a
    const float c_rest = fmaf(-0.5f, z, fmaf(z * z, c6, -fmaf(a, b, 0.5f * z_low)));        // cos - 1
    const float s = fmaf(scale, a, scale * s_rest), c = fmaf(scale, c_rest, scale);
    // cos(x + 90) = -sin x, sin(x + 90) = cos x
    const float x = (quarter & 1u) != 0u ? s : c, y = (quarter & 1u) != 0u ? c : s;
    *c_out = ((quarter + 1u) & 2u) != 0u ? -x : x;
    *s_out = (quarter & 2u) != 0u ? -y : y;
}

}  // namespace infllmv2
