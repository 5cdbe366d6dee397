// fp8_codes.h -- values as e4m3 codes with a power of two as the scale of a
// block.
//
//   scale = 2^ceil(log2(amax / 448)),  code = value / scale to the nearest e4m3
//
// A scale is held as its exponent + 127 (one byte), so it is also the scale
// operand of the matrix instructions.  The quotient is exact: codes differ
// from the nearest only where it would pass fp32's own range.
#pragma once

#include "host_device.h"

#include <stdint.h>

namespace moe {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTinyBits = 0x0d800000u;  // 2^-100: blocks below it count as zeros
constexpr int kUnitScale = 127;

// The scale byte of a block whose largest magnitude has these fp32 bits (an
// infinity or NaN in the block gives bits from kInfBits on).  448 = 1.75 2^8:
// the exponent less 8, and one more where the fraction passes 1.75.
MOE_HOST_DEVICE int fp8_scale_of(uint32_t top) {
    if (top >= kInfBits || top < kTinyBits) return kUnitScale;
    return static_cast<int>((top + 0x1fffffu) >> 23) - 8;
}

// The bits of 1 / scale.
MOE_HOST_DEVICE uint32_t fp8_inverse_bits(int scale) { return static_cast<uint32_t>(254 - scale) << 23; }

}  // namespace moe
