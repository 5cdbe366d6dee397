// codes.h -- fp32 values as 8-bit codes.
#pragma once

#include "host_device.h"

namespace moe {

// The code of x in a row whose largest magnitude is m >= 2^-100, inv = 1 / m
// rounded to fp32: 127 x / m to the nearest, ties to even, exactly.
//
// p + lo = 127 x exactly, r = p / m within one of the code.  e = p - r m is
// exact: a multiple of the smaller of the two units and below 2^24 of it (p <
// m leaves r in {0, 1}, and p - m between m / 2 and m is exact).  The quotient
// lies past the half way point on e's side where |e| + (lo towards it) > m /
// 2; the difference |e| - m / 2 is exact wherever it is close to zero, and
// adding lo keeps the sign.
MOE_HOST_DEVICE int code_of_f32(float x, float m, float inv) {
    const float p = 127.0f * x, lo = __builtin_fmaf(127.0f, x, -p);
    float r = __builtin_rintf(p * inv);
    const float e = __builtin_fmaf(-r, m, p);
    const float past = (__builtin_fabsf(e) - 0.5f * m) + (e < 0.0f ? -lo : lo);
    const bool odd = static_cast<int>(r) & 1;
    if (past > 0.0f || (past == 0.0f && odd)) r += __builtin_copysignf(1.0f, e);
    return static_cast<int>(r);
}

}  // namespace moe
