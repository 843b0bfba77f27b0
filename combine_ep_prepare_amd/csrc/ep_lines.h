// ep_lines.h -- weights streamed once for up to 16 rows of x, a wavefront at a
// time: the inner part of the products for few rows (ep_scaled.hip, ep_layer.hip).
//
// A handful of rows uses every weight once, so the weights' bytes bound it. A
// step of a wavefront is 128 bytes of each of a tile's columns (rows of the weight
// matrix). A load takes 8 columns x 128 bytes: whole lines, each asked for once,
// so that they can pass the caches by. A lane of a matrix instruction wants 16
// bytes of column lane % 16 instead, so the lines go from registers through a part
// of LDS that belongs to the wavefront alone, with no barrier: chunk c of column n
// at slot c ^ (n & 7). While a step is multiplied out of LDS, the next one's loads
// are in flight.
#pragma once

#include "ep_experts.h"
#include "ep_matrix.h"
#include "ep_scaled.h"

namespace epmi {

namespace {

// Eight e4m3 values to the payload type, exactly (both types hold them all).
template <int DT>
__device__ __forceinline__ row16_t widen8(uint32_t lo, uint32_t hi) {
  if constexpr (DT == EP_DTYPE_BF16) {
    return row16_t{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))};
  } else {
    return row16_t{
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true))};
  }
}

// Operands of a product for few rows.
enum Form {
  kPayload,   // weights and x of the payload type
  kScaled,    // weights and x in 8 bits, each with scales; multiplied as 16-bit values,
              // with fp32 sums (32 tokens by top-8 of 256, 7168 x 4096: 691 us, 690 with
              // the 8-bit instruction, which cuts them off; one expert of 16 rows, 4096 x
              // 4096: 10.7 against 9.9)
  kWeights8   // weights in 8 bits with scales, x of the payload type: a block's
              // sum is that of the e4m3 values themselves, and scaled in fp32
};

// Rows of x in fp16 with exponents: kExpGroup neighbours are kept as values of up to
// 2^15, the largest of them 2^14 at least, times a power of two of theirs, so that
// what fp32 holds is neither past fp16's range nor among its subnormals. The power is
// given by its exponent bits as an fp32 number, a byte. A byte of 1 or more and of 240
// or less: the power and its inverse are normal numbers.
constexpr int kExpGroup = 16;
__device__ __forceinline__ uint32_t exponent_for(float amax) {
  const uint32_t e = __float_as_uint(__builtin_fminf(amax, 0x1.fffffep127f)) >> 23;
  return (e > 15 ? e : 15) - 14;
}
__device__ __forceinline__ float power_of(uint32_t exponent) {
  return __uint_as_float(exponent << 23);
}
__device__ __forceinline__ float inverse_power_of(uint32_t exponent) {
  return __uint_as_float((254 - exponent) << 23);
}

// Eight fp16 values times 2^by, by <= 0, in two steps of half of it: each factor is
// an fp16 number down to 2^-44, where nothing is left of a value.
__device__ __forceinline__ row16_t lower8(row16_t v, int by) {
  by = by > -44 ? by : -44;
  const _Float16 f0 = __builtin_amdgcn_ldexph((_Float16)1.f, by >> 1);
  const _Float16 f1 = __builtin_amdgcn_ldexph((_Float16)1.f, by - (by >> 1));
  f16x8 h = __builtin_bit_cast(f16x8, v);
  h = h * f0 * f1;
  return __builtin_bit_cast(row16_t, h);
}

// A tile has COLS columns in two halves, which may lie apart (gate and up rows).
// EXPS: rows of x with exponents. A step's are brought to the largest one of its row,
// whose power the step's sums take.
template <int F, int DT, int COLS, bool EXPS = false>
struct Lines {
  static constexpr int kSize = F == kPayload ? 2 : 1;       // bytes of a weight
  static constexpr int kStep = 128 / kSize;                 // values of k
  static constexpr int kLoads = COLS / 8;
  static constexpr int kNF = COLS / 16;                     // blocks of 16 columns
  static constexpr int kX = F == kWeights8 ? 4 : 2;         // 16-byte parts of x
  static constexpr int kXSize = F == kScaled ? 1 : 2;
  static constexpr int kScales = F == kPayload ? 0 : F == kScaled ? 1 : kNF;
  static constexpr int kExpWords = EXPS ? kStep / kExpGroup / 4 : 0;   // of a step and row
  static constexpr int kLds = COLS * 128;
  static constexpr int kSumRow = COLS + 4;                  // floats of a row of sums
  static_assert(16 * kSumRow * 4 <= kLds, "the sums fit the weights' place");
  static_assert(!EXPS || (DT == EP_DTYPE_FP16 && F != kScaled), "rows of fp16 values");

  struct Source {
    const char* w[2];            // first column of either half, the same in all lanes
    int32_t cols[2];             // columns of either half that there are, multiples of 8
    const char* x;               // the lane's row of x
    const float* x_scales;       // its scales (kScaled)
    const uint8_t* x_exps;       // its exponents (EXPS), those of whole steps
    const float* w_scales[kScales > 0 ? kScales : 1];   // of the lane's columns
  };

  row16_t w[kLoads];
  row16_t x[kX];
  float scale[kScales > 0 ? kScales : 1];
  float x_scale;
  uint32_t exps[kExpWords > 0 ? kExpWords : 1];

  // The k, in the step, of part p of this lane's x: the same as that of the
  // weights that multiply() reads beside it.
  __device__ static __forceinline__ int32_t input(int p) {
    const int q = lane_id() >> 4;
    if constexpr (F == kPayload) return 32 * p + 8 * q;
    if constexpr (F == kScaled) return 64 * p + 16 * q;
    return 64 * (p / 2) + 16 * q + 8 * (p % 2);
  }

  // Loads of the step that starts at k0. In one that passes the end of the rows
  // (PART) a lane whose bytes are not there reads the rows' start and takes it
  // out again, of the weights and of x, whatever that holds.
  template <bool PART>
  __device__ __forceinline__ void load_weights(const Source& s, int32_t k0, int32_t K) {
    const int lane = lane_id();
    const uint32_t w_row = (uint32_t)K * kSize;
    const int chunk = (lane & 7) ^ (lane >> 3);
    const bool in = !PART || k0 + chunk * (kStep / 8) < K;
    const uint32_t at = (uint32_t)(lane >> 3) * w_row + (in ? (uint32_t)(k0 * kSize + chunk * 16) : 0u);
    static_for<kLoads>([&](auto j) {
      constexpr int half = j / (kLoads / 2), jj = j % (kLoads / 2);
      const char* column = s.w[half] + (jj * 8 < s.cols[half] ? jj * 8 * (int64_t)w_row : 0);
      w[j] = __builtin_nontemporal_load(reinterpret_cast<const row16_t*>(column + at));
      if constexpr (PART) w[j] = in ? w[j] : row16_t{0, 0, 0, 0};
    });
  }
  template <bool PART>
  __device__ __forceinline__ void load_x(const Source& s, int32_t k0, int32_t K) {
    static_for<kX>([&](auto p) {
      const int32_t k = k0 + input(p);
      const bool have = !PART || k < K;
      x[p] = *reinterpret_cast<const row16_t*>(s.x + (have ? (int64_t)k * kXSize : 0));
      if constexpr (PART) x[p] = have ? x[p] : row16_t{0, 0, 0, 0};
    });
    if constexpr (F != kPayload) {
      const int32_t block = k0 / kScaleBlock;
      static_for<kScales>([&](auto i) { scale[i] = s.w_scales[i][block]; });
      if constexpr (F == kScaled) x_scale = s.x_scales[block];
    }
    static_for<kExpWords>([&](auto i) {
      const int32_t group = k0 / kExpGroup + i * 4;
      exps[i] = *reinterpret_cast<const uint32_t*>(s.x_exps + group);
      if constexpr (PART) {
        // past the row's groups nothing was written
        const int32_t have = pieces(K, kExpGroup) - group;
        exps[i] &= have >= 4 ? 0xFFFFFFFFu : have <= 0 ? 0u : (1u << (have * 8)) - 1;
      }
    });
  }
  // The step's x to the largest of its exponents, which it returns.
  template <int WORDS>
  __device__ static __forceinline__ uint32_t level(row16_t (&xs)[kX],
                                                   const uint32_t (&ex)[WORDS]) {
    uint32_t most = 0;
    static_for<WORDS * 4>([&](auto i) {
      const uint32_t e = (ex[i / 4] >> (i % 4 * 8)) & 0xFF;
      most = e > most ? e : most;
    });
    static_for<kX>([&](auto p) {
      const int group = input(p) / kExpGroup;
      const uint32_t word = ex[p * WORDS / kX];
      const uint32_t own = (word >> (group % 4 * 8)) & 0xFF;
      xs[p] = lower8(xs[p], (int)own - (int)most);
    });
    return most;
  }
  template <bool PART>
  __device__ __forceinline__ void load(const Source& s, int32_t k0, int32_t K) {
    load_weights<PART>(s, k0, K);
    load_x<PART>(s, k0, K);
  }

  // The loaded weights into the wavefront's LDS. Its lanes write and read it in
  // program order; the fences keep the compiler to it.
  __device__ __forceinline__ void put(char* lds) const {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    static_for<kLoads>([&](auto j) {
      *reinterpret_cast<row16_t*>(lds + j * 1024 + lane_id() * 16) = w[j];
    });
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

  // Multiplies the loaded step; with MORE, the whole step from k1 on is asked for
  // as soon as the registers are free.
  template <bool MORE>
  __device__ __forceinline__ void step(char* lds, const Source& s, int32_t k1, int32_t K,
                                       f32x4 (&acc)[kNF]) {
    put(lds);
    row16_t xs[kX];
    static_for<kX>([&](auto p) { xs[p] = x[p]; });
    float sc[kScales > 0 ? kScales : 1];
    static_for<kScales>([&](auto i) { sc[i] = F == kScaled ? scale[i] * x_scale : scale[i]; });
    float power = 1.f;
    uint32_t ex[kExpWords > 0 ? kExpWords : 1];
    static_for<kExpWords>([&](auto i) { ex[i] = exps[i]; });
    if constexpr (MORE) load<false>(s, k1, K);
    if constexpr (EXPS) power = power_of(level(xs, ex));
    const int lane = lane_id(), q = lane >> 4, i16 = lane & 15;
    row16_t xw[F == kScaled ? 4 : 1];
    if constexpr (F == kScaled) {
      static_for<4>([&](auto p) {
        xw[p] = widen8<DT>(xs[p / 2][p % 2 * 2], xs[p / 2][p % 2 * 2 + 1]);
      });
    }
    const char* mine = lds + i16 * 128;
    const int slot0 = (q ^ (i16 & 7)) << 4, slot1 = ((4 + q) ^ (i16 & 7)) << 4;
    static_for<kNF>([&](auto j) {
      const row16_t a = *reinterpret_cast<const row16_t*>(mine + j * 2048 + slot0);
      const row16_t b = *reinterpret_cast<const row16_t*>(mine + j * 2048 + slot1);
      if constexpr (F == kPayload && !EXPS) {
        acc[j] = mma16<DT>(a, xs[0], acc[j]);
        acc[j] = mma16<DT>(b, xs[1], acc[j]);
      } else {
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
        if constexpr (F == kPayload) {
          part = mma16<DT>(a, xs[0], part);
          part = mma16<DT>(b, xs[1], part);
        } else {
          static_for<4>([&](auto p) {
            const row16_t& w8 = p < 2 ? a : b;
            row16_t xp;
            if constexpr (F == kScaled) xp = xw[p]; else xp = xs[p];
            part = mma16<DT>(widen8<DT>(w8[p % 2 * 2], w8[p % 2 * 2 + 1]), xp, part);
          });
        }
        // the sums of a lane are those of its own row of x
        float by = power;
        if constexpr (F != kPayload) by = EXPS ? sc[j] * power : sc[F == kScaled ? 0 : j.value];
        static_for<4>([&](auto c) {
          acc[j][c.value] = __builtin_fmaf(by, part[c.value], acc[j][c.value]);
        });
      }
    });
  }

  // All steps of a tile that are this wavefront's: every `waves`-th of them,
  // the first of which, if whole, has been asked for.
  __device__ __forceinline__ void steps(char* lds, const Source& s, int wave, int waves, int32_t K,
                                        f32x4 (&acc)[kNF]) {
    const int32_t full = K / kStep, stride = waves * kStep;
    if (wave < full) {
      int32_t k = wave * kStep;
      for (; k + stride < full * kStep; k += stride) step<true>(lds, s, k + stride, K, acc);
      step<false>(lds, s, 0, K, acc);
    }
    if (full * kStep < K && wave == full % waves) {
      load<true>(s, full * kStep, K);
      step<false>(lds, s, 0, K, acc);
    }
  }
  __device__ __forceinline__ void first(const Source& s, int wave, int32_t K) {
    if (wave < K / kStep) load<false>(s, wave * kStep, K);
  }

  // The wavefront's sums into its LDS: [row][column] of kSumRow floats.
  __device__ static __forceinline__ void put_sums(char* lds, const f32x4 (&acc)[kNF]) {
    const int lane = lane_id();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    static_for<kNF>([&](auto j) {
      *reinterpret_cast<f32x4*>(lds + ((lane & 15) * kSumRow + j * 16 + (lane >> 4) * 4) * 4) =
          acc[j];
    });
  }
  // Four columns from n on of row m, added up over the block's wavefronts.
  template <int WAVES>
  __device__ static __forceinline__ f32x4 sum_of(const char* mem, int m, int n) {
    const char* p = mem + (m * kSumRow + n) * 4;
    f32x4 sum = *reinterpret_cast<const f32x4*>(p);
    static_for<WAVES - 1>([&](auto v) {
      sum += *reinterpret_cast<const f32x4*>(p + (v + 1) * kLds);
    });
    return sum;
  }
};

}  // namespace

}  // namespace epmi
