// ep_quantise.h -- device side of ep_scaled.h: rounding to e4m3 with a scale for
// a block of values that a group of lanes holds.
#pragma once

#include "ep_device.h"
#include "ep_scaled.h"

namespace epmi {

namespace {

__device__ __forceinline__ float finite_magnitude(float v) {
  const float m = __builtin_fabsf(v);
  return m < __builtin_inff() ? m : 0.f;   // false for a NaN too
}

// The largest of m over aligned groups of LANES lanes (a power of two up to 32),
// in every lane of the group.
template <int LANES>
__device__ __forceinline__ float group_max(float m) {
  static_for<5>([&](auto i) {
    if constexpr ((1 << i) < LANES) m = __builtin_fmaxf(m, __shfl_xor(m, 1 << i, kWave));
  });
  return m;
}

// A block's scale, and what its values are multiplied by: the reciprocal of the
// scale but for its rounding, so that q is off the definition's quotient only
// where that lies next to the middle of two e4m3 values.
struct BlockScale {
  float scale, by;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  const float m = __builtin_fmaxf(amax, kLeastAmax);
  return BlockScale{m / kE4m3Max, kE4m3Max / m};
}

// Four values to e4m3, to nearest, ties to even. An infinity times `by` stays
// one and a NaN a NaN; both become e4m3's NaN (0x7F, which the conversion may
// give with either sign).
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d) {
  // an infinity would be cut off at 448, were the conversion to saturate
  auto nan = [](float v) { return __builtin_fabsf(v) < __builtin_inff() ? v : __builtin_nanf(""); };
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(nan(a), nan(b), 0, false);
  q = __builtin_amdgcn_cvt_pk_fp8_f32(nan(c), nan(d), q, true);
  return (uint32_t)q;
}

}  // namespace

}  // namespace epmi
