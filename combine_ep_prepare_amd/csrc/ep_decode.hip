// ep_decode.hip -- the grouped product for few rows per expert (decoding),
// with 16-bit weights or with 4-bit weights, a scale and a zero point per
// group of inputs:
//
//   out[r, n] = sum_h W[e][n, h] x[r, h]
//   W[e][n, h] = (q[e][n, h] - z[e][n, h / G]) * s[e][n, h / G]   (4 bits)
//
// A handful of rows uses every weight once, so the weights' bytes bound it:
// they go from memory straight to registers, 16 bytes a lane, and into matrix
// instructions whose other operand is up to 16 rows of x.
//
// 4-bit weights. A weight's four bits are put into the mantissa of a constant B,
// one mask-and-or for two of them and no conversion, and what leaves B again
// must not cost the sum its bits: most weights lie near their zero point, where
// a group's sum of (B + q) x is many times its sum of (q - z) x.
//   fp16: B = 1024, and a packed subtraction of B + z gives the operand q - z,
//   exact for every byte z (both are whole numbers below 2048). The group's sum is
//   that of the definition, infinite x included.
//   bf16 has no packed subtraction. The operand is B + q with the least B whose
//   mantissa holds four more bits, 16, and the group's fp32 sum starts at what
//   the offsets will add,
//     sum over the group of (q - z) x = -(B + z) S + sum (B + q) x,
//   S = sum of x over the group by the same instructions with a constant weight.
//   On values of 8 bits the sums stay exact over four powers of two of x (11 bits
//   of x, 5 of a weight, 7 for the 128 of a group, of 24). A group that starts at
//   zero and is corrected behind takes four more instructions for each 16 columns
//   (batch of 32, 256 experts: 453 us against 445).
// The scale is applied to the group's fp32 sum; no weight is rounded.

#include "ep_choice.h"
#include "ep_experts.h"

namespace epmi {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;             // wavefronts of a block: they split k
constexpr int kThreads = kWaves * kWave;
constexpr int kNF = 4;                // 16-column blocks of a wavefront
constexpr int kCols = 16 * kNF;       // columns of a tile
constexpr int kRowTile = 16;          // rows of a tile
constexpr int kLdsRow = kCols + 4;    // floats of a row of kCols in LDS

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

// B in both halves of a word, and the place of the four bits in a half.
template <int DT>
struct Offset {
  static constexpr float kValue = DT == EP_DTYPE_BF16 ? 16.f : 1024.f;
  // the weight of S: -(B + 8) in both halves where 8 is the zero point, else 1
  static constexpr uint32_t kStart[2] = {0xC1C0C1C0u, 0x3F803F80u};   // bf16
  static constexpr uint32_t kBits = DT == EP_DTYPE_BF16 ? 0x41804180u : 0x64006400u;
  static constexpr int kShift = DT == EP_DTYPE_BF16 ? 3 : 0;
};

// -(B + z) in both halves, fp16.
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) { return (0xE400u + z) * 0x10001u; }

// Eight weights of a word as operands, in the order 0 4 1 5 2 6 3 7: q - z in
// fp16, with `zero` from minus_zero, B + q in bf16. `bits` is Offset::kBits from
// a vector register: with the mask in a scalar one, each pair is one mask-and-or
// (two constants cannot both be scalar).
template <int DT>
__device__ __forceinline__ row16_t spread(uint32_t w, uint32_t bits, uint32_t zero) {
  constexpr int kShift = Offset<DT>::kShift;
  constexpr uint32_t kMask = 0x000F000Fu << kShift;
  typedef _Float16 half2 __attribute__((ext_vector_type(2)));
  row16_t o;
  static_for<4>([&](auto i) {
    constexpr int right = 4 * i.value - kShift;
    uint32_t v = w;
    if constexpr (right > 0) v = w >> right;
    if constexpr (right < 0) v = w << -right;
    v = (v & kMask) | bits;
    if constexpr (DT == EP_DTYPE_FP16)
      v = __builtin_bit_cast(uint32_t,
                             __builtin_bit_cast(half2, v) + __builtin_bit_cast(half2, zero));
    o[i.value] = v;
  });
  return o;
}

// Eight 16-bit values of x put into the same order.
__device__ __forceinline__ row16_t interleave(row16_t v) {
  return row16_t{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
                 __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// The 4 x 4 transpose of words over the quarters of a wavefront: word t of
// quarter q becomes word q of quarter t.
__device__ __forceinline__ row16_t transpose_quarters(row16_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return row16_t{c[0], c[1], e[0], e[1]};
}

// A step of k for a wavefront: 128 bytes of each of the tile's 64 columns, i.e.
// 256 inputs of 4 bits or 64 of 16 bits, in two halves of 64 bytes.
//
// A weight load is 8 columns x 128 bytes: whole lines, each of them asked for
// once, so that they can bypass the caches' retention (nontemporal). A lane
// of a matrix instruction wants 16 bytes of column lane % 16 instead; loads
// of that shape touch 16 lines of 64 bytes and ran at 5.4 TB/s where these
// run at 6.8 (batch of 32, 256 experts, weights only). So the lines go from
// registers through a part of LDS that belongs to the wavefront alone, with
// no barrier: chunk c of column n at slot c ^ (n & 7).
// While a step is multiplied out of LDS, the next one's loads are in flight.
//
// The quarter q = lane / 16 picks the part of k. 4 bits: with G = 128 word t
// of quarter q is inputs 32 q + 8 t of the half; for smaller groups, whose
// sums must not mix, the words are transposed over the quarters first and
// word t of quarter q is inputs 32 t + 8 q. 16 bits: inputs 8 q of the half.
template <int DT, bool QUANT, int G, bool ZEROS>
struct Stream {
  static constexpr int kStep = QUANT ? 256 : 64;
  static constexpr int kHalf = kStep / 2;
  static constexpr int kParts = QUANT ? 4 : 1;           // matrix instructions of a half
  static constexpr int kGroups = QUANT ? kHalf / G : 1;  // groups of a half
  static constexpr int kPer = 4 / kGroups;               // 4 bits: parts of a group
  static constexpr int kRows = QUANT ? 2 * kGroups : 0;  // groups of a step
  static constexpr int kLoads = kCols / 8;
  static constexpr bool kExact = QUANT && DT == EP_DTYPE_FP16;   // operands q - z
  // LDS of a wavefront: the weights of a step (in the end its sums), then the
  // step's scales and zero points as [group][column]: -(B + z) as a float, or
  // minus_zero's word
  static constexpr int kLds = kCols * 128 + (ZEROS ? 2 : 1) * kRows * kLdsRow * 4;

  // Where a tile's operands start (the same for the whole block), and a
  // lane's row of x.
  struct Source {
    const char* w;
    const char* x;
    const uint16_t* scales;
    const uint8_t* zeros;
    uint32_t x_off;
    int32_t cols;
  };

  row16_t w[kLoads];
  row16_t x[kParts];                   // of the half that comes next
  // of column `lane`, as they lie in memory: a register holds two scales or
  // four zero points until the step's end
  uint32_t scale[QUANT ? kRows / 2 : 1];
  uint32_t zero[QUANT ? (kRows + 3) / 4 : 1];

  __device__ static __forceinline__ int32_t input(int half, int t) {
    const int q = lane_id() >> 4;
    return half * kHalf + (QUANT && G == 128 ? 32 * q + 8 * t : 32 * t + 8 * q);
  }

  // Loads of the step that starts at input k0. One that passes the end of the
  // row (PART) reads the row's start in place of what is not there and takes
  // it out again: x counts zero, and so do 16-bit weights and scales.
  template <bool PART>
  __device__ __forceinline__ void load_weights(const Source& s, int32_t k0, int32_t H) {
    const int lane = lane_id();
    const uint32_t w_row = QUANT ? H / 2 : H * 2;
    const int chunk = (lane & 7) ^ (lane >> 3);
    const bool in = !PART || k0 + chunk * (kStep / 8) < H;
    const uint32_t at = (uint32_t)(lane >> 3) * w_row + chunk * 16;
    const char* from = s.w + (QUANT ? k0 / 2 : k0 * 2);
    static_for<kLoads>([&](auto j) {
      const char* column = from + (j * 8 < s.cols ? j * 8 * (int64_t)w_row : 0);
      if constexpr (PART) column -= in ? 0 : (QUANT ? k0 / 2 : k0 * 2) + chunk * 16;
      w[j] = __builtin_nontemporal_load(reinterpret_cast<const row16_t*>(column + at));
      if constexpr (PART && !QUANT) w[j] = in ? w[j] : row16_t{0, 0, 0, 0};
    });
    if constexpr (QUANT) {
      const int32_t all = H / G, g0 = k0 / G;
      const int64_t row = (int64_t)(lane < s.cols ? lane : 0) * all + g0;
      if constexpr (PART) {
        static_for<kRows / 2>([&](auto g) { scale[g] = 0; });
        static_for<(kRows + 3) / 4>([&](auto g) { zero[g] = 0; });
        static_for<kRows>([&](auto g) {
          const bool have = g0 + g < all;
          if (have) scale[g / 2] |= (uint32_t)s.scales[row + g] << (g % 2 * 16);
          if constexpr (ZEROS)
            if (have) zero[g / 4] |= (uint32_t)s.zeros[row + g] << (g % 4 * 8);
        });
      } else {
        __builtin_memcpy(scale, s.scales + row, kRows * 2);
        if constexpr (ZEROS) __builtin_memcpy(zero, s.zeros + row, kRows);
      }
    }
  }
  template <bool PART>
  __device__ __forceinline__ void load_x(const Source& s, int half, int32_t k0, int32_t H) {
    static_for<kParts>([&](auto t) {
      const int32_t k = k0 + input(half, t);
      const bool in = !PART || k < H;
      const row16_t v =
          *reinterpret_cast<const row16_t*>(s.x + (s.x_off + (uint32_t)(in ? k : 0) * 2));
      x[t] = in ? v : row16_t{0, 0, 0, 0};
    });
  }

  // The loaded weights and scales into the wavefront's LDS. Its lanes write
  // and read it in program order; the fences keep the compiler to it.
  __device__ __forceinline__ void put(char* lds) const {
    const int lane = lane_id();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    static_for<kLoads>([&](auto j) {
      *reinterpret_cast<row16_t*>(lds + j * 1024 + lane * 16) = w[j];
    });
    if constexpr (QUANT) {
      float* scales = reinterpret_cast<float*>(lds + kCols * 128);
      float* zeros = scales + kRows * kLdsRow;
      static_for<kRows>([&](auto g) {
        const uint32_t sc = g % 2 ? scale[g / 2] >> 16 : scale[g / 2] & 0xFFFFu;
        scales[g * kLdsRow + lane] =
            DT == EP_DTYPE_BF16 ? __uint_as_float(sc << 16) : f16_to_f32(sc);
        if constexpr (ZEROS) {
          const uint32_t z = (zero[g / 4] >> (g % 4 * 8)) & 0xFFu;
          zeros[g * kLdsRow + lane] = kExact ? __uint_as_float(minus_zero(z))
                                             : -(Offset<DT>::kValue + (float)z);
        }
      });
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }

  // One half out of LDS; xs is its x, already interleaved for 4 bits.
  __device__ static __forceinline__ void multiply(const char* lds, int half,
                                                  const row16_t (&xs)[kParts], uint32_t bits,
                                                  f32x4 (&acc)[kNF]) {
    const int lane = lane_id(), q = lane >> 4, i16 = lane & 15;
    const char* mine = lds + i16 * 128 + (((half * 4 + q) ^ (i16 & 7)) << 4);
    if constexpr (!QUANT) {
      static_for<kNF>([&](auto j) {
        acc[j] = mma16<DT>(*reinterpret_cast<const row16_t*>(mine + j * 2048), xs[0], acc[j]);
      });
    } else {
      const float* scales = reinterpret_cast<const float*>(lds + kCols * 128);
      const float* zeros = scales + kRows * kLdsRow;
      // where operands hold B: S, the same in all four
      f32x4 start[kGroups];
      static_for<kGroups>([&](auto g) {
        start[g] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (!kExact) {
          constexpr uint32_t one = Offset<DT>::kStart[ZEROS];
          static_for<kPer>([&](auto u) {
            start[g] = mma16<DT>(row16_t{one, one, one, one}, xs[g * kPer + u], start[g]);
          });
        }
      });
      static_for<kNF>([&](auto j) {
        row16_t words = *reinterpret_cast<const row16_t*>(mine + j * 2048);
        if constexpr (G < 128) words = transpose_quarters(words);
        static_for<kGroups>([&](auto g) {
          // one group's operands at a time: read ahead for all blocks, the
          // scales alone would take more registers than a wavefront has
          __builtin_amdgcn_sched_barrier(0);
          const int row = (half * kGroups + g) * kLdsRow + j * 16;
          const f32x4 scale = *reinterpret_cast<const f32x4*>(scales + row + q * 4);
          uint32_t zero_word = minus_zero(8);
          f32x4 part = start[g];
          // several groups: one register each is enough to keep
          if constexpr (kGroups > 1)
            static_for<3>([&](auto c) { part[c.value + 1] = part[0]; });
          if constexpr (ZEROS && kExact) {   // of the lane's column of weights
            zero_word = __float_as_uint(zeros[row + i16]);
          } else if constexpr (ZEROS) {      // of its columns of sums
            const f32x4 zero = *reinterpret_cast<const f32x4*>(zeros + row + q * 4);
            static_for<4>([&](auto c) { part[c.value] *= zero[c.value]; });
          }
          static_for<kPer>([&](auto u) {
            constexpr int t = g.value * kPer + u.value;
            part = mma16<DT>(spread<DT>(words[t], bits, zero_word), xs[t], part);
          });
          static_for<4>([&](auto c) {
            acc[j][c.value] = __builtin_fmaf(scale[c.value], part[c.value], acc[j][c.value]);
          });
        });
      });
    }
  }

  // The first loads of a step from input k0 on: weights, x of its first half.
  template <bool PART>
  __device__ __forceinline__ void load(const Source& s, int32_t k0, int32_t H) {
    load_weights<PART>(s, k0, H);
    load_x<PART>(s, 0, k0, H);
  }
  // Multiplies the loaded step (from input k0 on; the one that passes the end of
  // the row with PART); with MORE the whole step from input k1 on is loaded as
  // registers get free. Loads come back in order: x of the second half is asked
  // for ahead of the next step's weights, which it must not wait for.
  template <bool PART, bool MORE>
  __device__ __forceinline__ void step(char* lds, const Source& s, int32_t k0, int32_t k1,
                                       int32_t H, uint32_t bits, f32x4 (&acc)[kNF]) {
    put(lds);
    row16_t xs[kParts];
    auto take_x = [&]() {
      static_for<kParts>([&](auto t) { xs[t] = QUANT ? interleave(x[t]) : x[t]; });
    };
    take_x();
    load_x<PART>(s, 1, k0, H);
    if constexpr (MORE) load_weights<false>(s, k1, H);
    multiply(lds, 0, xs, bits, acc);
    take_x();
    if constexpr (MORE) load_x<false>(s, 0, k1, H);
    multiply(lds, 1, xs, bits, acc);
  }
};

// Blocks (of one wavefront a SIMD) to a CU, by the registers that they leave a
// wavefront. The 4-bit form in the 128 of four spills, at twice the time. Three
// leave 168, which hold all of its instances but the bf16 one with groups of 32
// and zero points: that one keeps 6 registers in scratch, and ran 45.6 us against
// 49.1 with two blocks and none there (sixteen tokens, top-8 of 128, 2048 inputs,
// 1536 outputs). 16-bit weights with four against three ran 90 against 95 us (the
// same routing).
constexpr int blocks_per_cu(bool quant) { return quant ? 3 : 4; }

// Up to 16 rows of an expert by kCols columns a block step. The wavefronts
// take the steps of k in turn, so that the block reads 512 bytes of a column
// side by side, and add their sums in LDS at the end; by then each has the
// first loads of the block's next tile in flight.
template <int DT, bool QUANT, int G, bool ZEROS>
__global__ void __launch_bounds__(kThreads, blocks_per_cu(QUANT))
    few_rows_kernel(Dims d, HandleView hv, const char* __restrict__ x,
                    const char* __restrict__ w, const uint16_t* __restrict__ scales,
                    const uint8_t* __restrict__ zeros, uint16_t* __restrict__ out, int64_t N) {
  using S = Stream<DT, QUANT, G, ZEROS>;
  extern __shared__ __align__(16) char mem[];
  int32_t* tile_start = reinterpret_cast<int32_t*>(mem + kWaves * S::kLds);
  const int32_t my_rows = rows_of_thread(hv, d);
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t row_tiles =
      list_tiles<kThreads>(hv, d, kRowTile, my_rows, tile_start, tile_start + d.E + 1);
  const int64_t ct = (N + kCols - 1) / kCols, tiles = row_tiles * ct;
  const int32_t H = (int32_t)d.H;
  const int lane = lane_id(), i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  char* lds = mem + wave * S::kLds;
  uint32_t bits = Offset<DT>::kBits;
  asm("" : "+v"(bits));

  struct Place {
    typename S::Source src;
    int64_t out;   // first row and column of the tile in `out`
    int32_t rows;
  };
  auto place = [&](int64_t t) {
    // the row tiles of an expert are neighbours: they run at the same time, and
    // each reads the weights for itself
    const int e = __builtin_amdgcn_readfirstlane(
        expert_of_tile(tile_start, d.E, (int32_t)(t / ct)));
    const int64_t in_e = t - tile_start[e] * ct;
    const int32_t rts = tile_start[e + 1] - tile_start[e];
    const int32_t ni = __builtin_amdgcn_readfirstlane((int32_t)(in_e / rts));
    const int32_t m0 =
        __builtin_amdgcn_readfirstlane((int32_t)(in_e - (int64_t)ni * rts)) * kRowTile;
    const Segment s = segment_of(hv, d, e);
    const int64_t n0 = (int64_t)ni * kCols, column = (int64_t)e * N + n0;
    Place p;
    p.rows = s.rows - m0 < kRowTile ? s.rows - m0 : kRowTile;
    p.out = (s.row + m0) * N + n0;
    p.src.w = w + column * (QUANT ? H / 2 : H * 2);
    p.src.x = x + (s.row + m0) * H * 2;
    p.src.scales = QUANT ? scales + column * (H / G) : nullptr;
    p.src.zeros = ZEROS ? zeros + column * (H / G) : nullptr;
    p.src.x_off = (uint32_t)(i16 < p.rows ? i16 : p.rows - 1) * (uint32_t)(H * 2);
    p.src.cols = (int32_t)(N - n0 < kCols ? N - n0 : kCols);
    return p;
  };
  const int32_t full = H / S::kStep;                      // whole steps
  const int32_t first = wave * S::kStep, stride = kWaves * S::kStep;
  S s;
  auto load = [&](const Place& p) {
    if (wave < full) s.template load<false>(p.src, first, H);
  };
  Place next;
  if ((int64_t)blockIdx.x < tiles) {
    next = place(blockIdx.x);
    load(next);
  }
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Place cur = next;
    f32x4 acc[kNF];
    static_for<kNF>([&](auto j) { acc[j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    if (wave < full) {
      int32_t k = first;
      for (; k + stride < full * S::kStep; k += stride)
        s.template step<false, true>(lds, cur.src, k, k + stride, H, bits, acc);
      s.template step<false, false>(lds, cur.src, k, 0, H, bits, acc);
    }
    if (full * S::kStep < H && wave == kWaves - 1) {
      s.template load<true>(cur.src, full * S::kStep, H);
      s.template step<true, false>(lds, cur.src, full * S::kStep, 0, H, bits, acc);
    }
    if (t + gridDim.x < tiles) {
      next = place(t + gridDim.x);
      load(next);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    static_for<kNF>([&](auto j) {
      float* p = reinterpret_cast<float*>(lds) + i16 * kLdsRow + j * 16 + (lane >> 4) * 4;
      *reinterpret_cast<f32x4*>(p) = acc[j];
    });
    __syncthreads();
    // four columns of a row a thread
    const int m = threadIdx.x / (kCols / 4), n = threadIdx.x % (kCols / 4) * 4;
    if (m < cur.rows && n < cur.src.cols) {
      const char* p = mem + (m * kLdsRow + n) * 4;
      f32x4 sum = *reinterpret_cast<const f32x4*>(p);
      static_for<kWaves - 1>([&](auto v) {
        sum += *reinterpret_cast<const f32x4*>(p + (v + 1) * S::kLds);
      });
      u32x2 o;
      if constexpr (DT == EP_DTYPE_BF16) {
        o = u32x2{rne_bf16(sum[0]) | (rne_bf16(sum[1]) << 16),
                  rne_bf16(sum[2]) | (rne_bf16(sum[3]) << 16)};
      } else {
        o = u32x2{rne_f16(sum[0]) | (rne_f16(sum[1]) << 16),
                  rne_f16(sum[2]) | (rne_f16(sum[3]) << 16)};
      }
      *reinterpret_cast<u32x2*>(out + cur.out + m * N + n) = o;
    }
    __syncthreads();  // the sums are read before the next tile's weights
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

template <int DT, bool QUANT, int G, bool ZEROS>
hipError_t launch_few_rows(const Dims& d, const HandleView& hv, const void* x, const void* w,
                           const void* scales, const uint8_t* zeros, void* out, int64_t N,
                           int num_cus, hipStream_t stream) {
  const int64_t ct = (N + kCols - 1) / kCols;
  const int64_t routes = most_rows(d);
  int64_t blocks = (routes / kRowTile + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * blocks_per_cu(QUANT);
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  const size_t lds = kWaves * (size_t)Stream<DT, QUANT, G, ZEROS>::kLds +
                     sizeof(int32_t) * (size_t)(d.E + 1 + kWaves);
  few_rows_kernel<DT, QUANT, G, ZEROS><<<dim3((uint32_t)blocks), dim3(kThreads), lds, stream>>>(
      d, hv, static_cast<const char*>(x), static_cast<const char*>(w),
      static_cast<const uint16_t*>(scales), zeros, static_cast<uint16_t*>(out), N);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_few(const Dims& d, const HandleView& hv, const void* x, const void* w,
                              void* out, int64_t N, int num_cus, hipStream_t stream) {
  if (d.dtype == EP_DTYPE_FP16)
    return launch_few_rows<EP_DTYPE_FP16, false, 128, false>(d, hv, x, w, nullptr, nullptr, out,
                                                             N, num_cus, stream);
  return launch_few_rows<EP_DTYPE_BF16, false, 128, false>(d, hv, x, w, nullptr, nullptr, out, N,
                                                           num_cus, stream);
}

hipError_t launch_grouped_quant(const Dims& d, const HandleView& hv, const void* x,
                                const uint8_t* q, const void* scales, const uint8_t* zeros,
                                void* out, int64_t N, int32_t group, int num_cus,
                                hipStream_t stream) {
  auto go = [&](auto dt, auto g, auto z) {
    return launch_few_rows<decltype(dt)::value, true, decltype(g)::value, decltype(z)::value>(
        d, hv, x, q, scales, zeros, out, N, num_cus, stream);
  };
  auto with_zeros = [&](auto dt, auto g) {
    return zeros ? go(dt, g, std::true_type{}) : go(dt, g, std::false_type{});
  };
  auto with_group = [&](auto dt) {
    switch (group) {
      case 32: return with_zeros(dt, std::integral_constant<int, 32>{});
      case 64: return with_zeros(dt, std::integral_constant<int, 64>{});
      default: return with_zeros(dt, std::integral_constant<int, 128>{});
    }
  };
  if (d.dtype == EP_DTYPE_FP16) return with_group(std::integral_constant<int, EP_DTYPE_FP16>{});
  return with_group(std::integral_constant<int, EP_DTYPE_BF16>{});
}

}  // namespace epmi
