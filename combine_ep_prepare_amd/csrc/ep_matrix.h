// ep_matrix.h -- vector types of the matrix instructions, the product of 16 x 16 x 32
// values of 16 bits, and the rounding of four sums, shared by the products.
#pragma once

#include "ep_device.h"

namespace epmi {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// acc += n m: 16 columns (rows of the weight matrix) by 16 rows of x, 8 values of k a
// lane; a lane gets four consecutive columns of row lane % 16.
template <int DT>
__device__ __forceinline__ f32x4 mma16(row16_t n, row16_t m, f32x4 acc) {
  if constexpr (DT == EP_DTYPE_BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, n), __builtin_bit_cast(bf16x8, m), acc, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(
        __builtin_bit_cast(f16x8, n), __builtin_bit_cast(f16x8, m), acc, 0, 0, 0);
  }
}

// Four results rounded to 16 bits.
template <int DT>
__device__ __forceinline__ u32x2 round4(f32x4 v) {
  if constexpr (DT == EP_DTYPE_BF16) {
    return u32x2{rne_bf16(v[0]) | (rne_bf16(v[1]) << 16),
                 rne_bf16(v[2]) | (rne_bf16(v[3]) << 16)};
  } else {
    return u32x2{rne_f16(v[0]) | (rne_f16(v[1]) << 16), rne_f16(v[2]) | (rne_f16(v[3]) << 16)};
  }
}

}  // namespace

}  // namespace epmi
