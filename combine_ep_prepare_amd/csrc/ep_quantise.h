// ep_quantise.h -- device side of ep_scaled.h: rounding to e4m3 with a scale for
// a block of values that a group of lanes holds.
#pragma once

#include "ep_device.h"
#include "ep_scaled.h"

namespace epmi {

namespace {

// The largest of m, 0 or more, over aligned groups of LANES lanes (16 or 32), in
// every lane of the group. Numbers of that sign are in the order of their bits; a
// lane's neighbours come within the instruction that compares them.
template <int LANES>
__device__ __forceinline__ float group_max(float m) {
  static_assert(LANES == 16 || LANES == 32, "16-bit or fp32 rows");
  uint32_t v = __float_as_uint(m);
  auto with = [&](auto order) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, order.value, 0xf, 0xf, true);
    v = o > v ? o : v;
  };
  using std::integral_constant;
  with(integral_constant<int, 0xB1>{});    // lanes 1, 0, 3, 2 of four
  with(integral_constant<int, 0x4E>{});    // 2, 3, 0, 1
  with(integral_constant<int, 0x141>{});   // eight backwards
  with(integral_constant<int, 0x140>{});   // sixteen backwards
  if constexpr (LANES == 32) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, 16, kWave);
    v = o > v ? o : v;
  }
  return __uint_as_float(v);
}

// A block's scale, and its reciprocal, which the values are multiplied by: q is off
// the definition's quotient only where that lies next to the middle of two e4m3
// values. Each is a product or a reciprocal with the rest that it leaves put back,
// good to its last bit; between 2^-100 and 2^120 nothing overflows or is subnormal.
struct BlockScale {
  float scale, by;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  constexpr float kInverse = 1.f / kE4m3Max;
  const float m = __builtin_fmaxf(amax, kLeastAmax);
  const float q = m * kInverse;
  const float scale = __builtin_fmaf(__builtin_fmaf(-kE4m3Max, q, m), kInverse, q);
  const float r = __builtin_amdgcn_rcpf(scale);
  return BlockScale{scale, __builtin_fmaf(__builtin_fmaf(-scale, r, 1.f), r, r)};
}

// NV values of a block, of which a group of LANES lanes holds NV each, to e4m3, four
// to a word; returns the scale. Called by whole groups. Values that are not finite
// are looked for by the wavefront, in scalars, and taken apart only where there are
// any: apart from that a value costs its maximum, half a comparison, a product and
// half a conversion.
template <int LANES, int NV>
__device__ __forceinline__ float quantise(const float (&y)[NV], uint32_t (&q)[NV / 4]) {
  float amax = 0.f, v[NV];
  uint64_t odd = 0;
  static_for<NV / 2>([&](auto i) {
    odd |= wave_ballot(__builtin_isunordered(y[2 * i], y[2 * i + 1]));
  });
  static_for<NV>([&](auto i) {
    v[i] = y[i];
    amax = __builtin_fmaxf(amax, __builtin_fabsf(y[i]));   // past a NaN
  });
  odd |= wave_ballot(amax == __builtin_inff());
  if (odd != 0) {
    amax = 0.f;
    static_for<NV>([&](auto i) {
      // both become e4m3's NaN: an infinity could be cut off at 448
      const bool fine = __builtin_fabsf(y[i]) < __builtin_inff();
      v[i] = fine ? y[i] : __builtin_nanf("");
      amax = __builtin_fmaxf(amax, fine ? __builtin_fabsf(y[i]) : 0.f);
    });
  }
  const BlockScale b = block_scale(group_max<LANES>(amax));
  static_for<NV / 4>([&](auto i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * b.by, v[4 * i + 1] * b.by, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * b.by, v[4 * i + 3] * b.by, w, true);
    q[i] = (uint32_t)w;
  });
  return b.scale;
}

// A lane's 8-bit values, four or eight of them, past the caches.
template <int W>
__device__ __forceinline__ void store_bytes(uint8_t* to, const uint32_t (&q)[W]) {
  if constexpr (W == 2) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u32x2{q[0], q[1]}, reinterpret_cast<u32x2*>(to));
  } else {
    static_assert(W == 1, "16-bit or fp32 rows");
    __builtin_nontemporal_store(q[0], reinterpret_cast<uint32_t*>(to));
  }
}

}  // namespace

}  // namespace epmi
