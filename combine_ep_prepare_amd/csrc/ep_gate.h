// ep_gate.h -- the sigmoid of the gated activation, and the rounding of eight
// results at a time, shared by the kernels that compute activations or norms.
#pragma once

#include "ep_device.h"

namespace epmi {

namespace {

// What the results take from a gate g. With e = exp(-|g|) and r = 1 / (1 + e),
//   s = 1 / (1 + exp(-g)) = p^2 r and 1 - s = q, where
//   p = 1, q = e r for g >= 0 and p = sqrt(e), q = r for g < 0:
// no exponential overflows, 1 - s does not cancel, and s enters a product as
// one p a factor, so that a sigmoid below fp32's range still counts: a gate of
// -88 gives silu(g) = -5e-37. p is a normal number down to g = -174, past which
// it is 0.
struct Gate {
  float p, q, r;
};

// The exponent |g| log2(e) / 2 of p is rounded, which takes p off by up to
// |g| / 2 units of 2^-24: nothing to a 16-bit result (a gate of 174 makes 2^-16
// of it in s). EXACT, for fp32, carries what the rounding and the constant
// leave out into p and refines the reciprocal by a step: s is then within 20
// units of 2^-24 of its value at any g, in the time that the rows' bytes take
// anyway (8192 rows by top-2, 4096 values out: 146 us with it and without).
// SHORT, for the kernel that the arithmetic bounds, rounds 1 + e once.
template <bool EXACT, bool SHORT = false>
__device__ __forceinline__ Gate gate_of(float g) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  constexpr float kHalfLn2 = 0.34657359027997265f;
  Gate o;
  float root;   // sqrt(e)
  if constexpr (EXACT) {
    // past 400 p is 0, and an infinite g would make the rest a NaN
    const float x = __builtin_fminf(__builtin_fabsf(g), 400.f);
    const float a = x * kHi;
    const float rest = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -a));
    root = __builtin_amdgcn_exp2f(a * -0.5f);
    root = __builtin_fmaf(root, rest * -kHalfLn2, root);
  } else {
    root = __builtin_amdgcn_exp2f(__builtin_fabsf(g) * (-0.5f * kHi));
  }
  const float e = root * root, d = SHORT ? __builtin_fmaf(root, root, 1.f) : 1.f + e;
  o.r = __builtin_amdgcn_rcpf(d);
  if constexpr (EXACT) o.r = __builtin_fmaf(__builtin_fmaf(-d, o.r, 1.f), o.r, o.r);
  o.p = g < 0.f ? root : 1.f;
  o.q = g < 0.f ? o.r : e * o.r;
  return o;
}

// Rounds like Payload::pack; where no lane has a NaN, by the hardware's packed
// conversions.
template <int DT, int N>
__device__ __forceinline__ row16_t pack(const float (&o)[N]) {
  if constexpr (DT != EP_DTYPE_FP32) {
    bool nan = false;
    static_for<N / 2>([&](auto j) { nan |= __builtin_isunordered(o[2 * j], o[2 * j + 1]); });
    if (wave_ballot(nan) == 0) {
      typedef std::conditional_t<DT == EP_DTYPE_BF16, __bf16, _Float16> half;
      typedef half half2 __attribute__((ext_vector_type(2)));
      typedef float float2v __attribute__((ext_vector_type(2)));
      row16_t v;
      static_for<4>([&](auto j) {
        float2v f = {o[2 * j], o[2 * j + 1]};
        // the fp32 results stand as they are: no fusing of the last product
        // with the conversion, which would skip its rounding
        asm("" : "+v"(f));
        v[j.value] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, half2));
      });
      return v;
    }
  }
  return Payload<DT>::pack(o);
}

}  // namespace

}  // namespace epmi
