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
// 4-bit weights. A weight enters the matrix instruction as the exact value
// B + q, B = 128 in bf16 and 1024 in fp16, which is the word's four bits put
// under the exponent of B: one mask-and-or for two weights, no conversion.
// With S = sum of x over a group (the same instructions with a weight of 1),
//   sum over the group of (q - z) s x = s * (sum (B + q) x - (B + z) S)
// in fp32: no weight is rounded, and the offset costs about log2(2 B / 15)
// of the 24 bits of the group's sum, which leaves more than a 16-bit result
// holds.

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
constexpr int kStageK = 8192;         // inputs whose scales are staged at once
constexpr int kRedRow = kCols + 4;    // floats of a row of partial sums in LDS

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

template <int DT>
struct Offset {
  static constexpr float kValue = DT == EP_DTYPE_BF16 ? 128.f : 1024.f;
  static constexpr uint32_t kBits = DT == EP_DTYPE_BF16 ? 0x43004300u : 0x64006400u;
  static constexpr uint32_t kOnes = DT == EP_DTYPE_BF16 ? 0x3F803F80u : 0x3C003C00u;
};

// Eight weights of a word as offset values, in the order 0 4 1 5 2 6 3 7.
template <int DT>
__device__ __forceinline__ row16_t spread(uint32_t w) {
  constexpr uint32_t kMask = 0x000F000Fu;
  return row16_t{(w & kMask) | Offset<DT>::kBits, ((w >> 4) & kMask) | Offset<DT>::kBits,
                 ((w >> 8) & kMask) | Offset<DT>::kBits,
                 ((w >> 12) & kMask) | Offset<DT>::kBits};
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

// The inputs of one step of k for a lane. A lane works on column lane % 16 of
// each block of weights and row lane % 16 of x; its quarter q = lane / 16
// picks the part of k.
// 4 bits: a step is 128 inputs, one 16-byte load of 32 weights a lane and
// block. With G = 128 word t of quarter q is inputs 32 q + 8 t; for smaller
// groups, whose sums must not mix, the words are transposed over the quarters
// first and word t of quarter q is inputs 32 t + 8 q.
// 16 bits: a step is 64 inputs, two loads a lane and block.
template <bool QUANT>
struct Step {
  static constexpr int kStep = QUANT ? 128 : 64;
  static constexpr int kParts = QUANT ? 4 : 2;   // matrix instructions of a block
  static constexpr int kWords = QUANT ? 1 : 2;   // 16-byte loads of a block
  row16_t w[kNF][kWords];
  row16_t x[kParts];
};

// Where a lane reads: the tile's weights and rows (the same for the block)
// and its own column of each block and row, as offsets from there.
struct Source {
  const char* w;
  const char* x;
  uint32_t w_off[kNF];
  uint32_t x_off;
};

template <int DT, bool QUANT, int G, bool ZEROS>
struct Tile {
  using S = Step<QUANT>;
  static constexpr int kStep = S::kStep;
  static constexpr int kGroups = QUANT ? kStep / G : 1;  // groups of a step
  static constexpr int kPer = 4 / kGroups;               // 4 bits: parts of a group

  // Loads the step that starts at input k0. Past the end of the row it reads
  // the row's start instead; finish() takes those values out.
  __device__ static __forceinline__ void load(S& s, const Source& src, int32_t k0, int32_t H) {
    const int q = lane_id() >> 4;
    if constexpr (QUANT) {
      const int32_t k = k0 + 32 * q;
      const uint32_t at = (k < H ? k : 0) / 2;
      static_for<kNF>([&](auto j) {
        s.w[j][0] = __builtin_nontemporal_load(
            reinterpret_cast<const row16_t*>(src.w + (src.w_off[j] + at)));
      });
    } else {
      static_for<S::kWords>([&](auto t) {
        const int32_t k = k0 + 32 * t + 8 * q;
        const uint32_t at = (k < H ? k : 0) * 2;
        static_for<kNF>([&](auto j) {
          s.w[j][t] = __builtin_nontemporal_load(
              reinterpret_cast<const row16_t*>(src.w + (src.w_off[j] + at)));
        });
      });
    }
    static_for<S::kParts>([&](auto t) {
      const int32_t k = input(k0, t);
      const uint32_t at = (k < H ? k : 0) * 2;
      s.x[t] = *reinterpret_cast<const row16_t*>(src.x + (src.x_off + at));
    });
  }

  // The input that part t of a step starts at, for this lane.
  __device__ static __forceinline__ int32_t input(int32_t k0, int t) {
    const int q = lane_id() >> 4;
    return k0 + (QUANT && G == 128 ? 32 * q + 8 * t : 32 * t + 8 * q);
  }

  // Inputs past the end of the row count nothing: x is zero there, and so
  // are 16-bit weights.
  __device__ static __forceinline__ void finish(S& s, int32_t k0, int32_t H) {
    if (k0 + kStep <= H) return;
    const row16_t zero = {0, 0, 0, 0};
    static_for<S::kParts>([&](auto t) {
      const bool in = input(k0, t) < H;
      s.x[t] = in ? s.x[t] : zero;
      if constexpr (!QUANT) {
        static_for<kNF>([&](auto j) { s.w[j][t] = in ? s.w[j][t] : zero; });
      }
    });
  }

  // scales, zeros: the step's first group in LDS, [group][column].
  __device__ static __forceinline__ void multiply(S& s, int32_t k0, int32_t H,
                                                  const uint16_t* scales, const uint8_t* zeros,
                                                  f32x4 (&acc)[kNF]) {
    finish(s, k0, H);
    if constexpr (!QUANT) {
      static_for<S::kParts>([&](auto t) {
        static_for<kNF>([&](auto j) { acc[j] = mma16<DT>(s.w[j][t], s.x[t], acc[j]); });
      });
    } else {
      const int q = lane_id() >> 4;
      row16_t xs[4];
      f32x4 sum[kGroups];
      constexpr uint32_t one = Offset<DT>::kOnes;
      static_for<4>([&](auto t) { xs[t] = interleave(s.x[t]); });
      static_for<kGroups>([&](auto g) {
        sum[g] = f32x4{0.f, 0.f, 0.f, 0.f};
        static_for<kPer>([&](auto u) {
          sum[g] = mma16<DT>(row16_t{one, one, one, one}, xs[g * kPer + u], sum[g]);
        });
      });
      static_for<kNF>([&](auto j) {
        const row16_t words = G == 128 ? s.w[j][0] : transpose_quarters(s.w[j][0]);
        static_for<kGroups>([&](auto g) {
          // one group's operands at a time: read ahead for all blocks, the
          // scales alone would take more registers than a wavefront has
          __builtin_amdgcn_sched_barrier(0);
          const int at = g * kCols + j * 16 + q * 4;
          const u32x2 sc = *reinterpret_cast<const u32x2*>(scales + at);
          f32x4 scale, zero;
          if constexpr (DT == EP_DTYPE_BF16) {
            scale = f32x4{bf16_lo(sc[0]), bf16_hi(sc[0]), bf16_lo(sc[1]), bf16_hi(sc[1])};
          } else {
            scale = f32x4{f16_to_f32(sc[0] & 0xFFFFu), f16_to_f32(sc[0] >> 16),
                          f16_to_f32(sc[1] & 0xFFFFu), f16_to_f32(sc[1] >> 16)};
          }
          if constexpr (ZEROS) {
            const uint32_t z = *reinterpret_cast<const uint32_t*>(zeros + at);
            static_for<4>([&](auto c) {
              zero[c.value] = Offset<DT>::kValue + (float)((z >> (8 * c.value)) & 255u);
            });
          } else {
            static_for<4>([&](auto c) { zero[c.value] = Offset<DT>::kValue + 8.f; });
          }
          f32x4 part = {0.f, 0.f, 0.f, 0.f};
          static_for<kPer>([&](auto u) {
            constexpr int t = g.value * kPer + u.value;
            part = mma16<DT>(spread<DT>(words[t]), xs[t], part);
          });
          static_for<4>([&](auto c) {
            const float v = __builtin_fmaf(-zero[c.value], sum[g][0], part[c.value]);
            acc[j][c.value] = __builtin_fmaf(scale[c.value], v, acc[j][c.value]);
          });
        });
      });
    }
  }
};

// Blocks (of one wavefront a SIMD) that the registers allow: small groups
// keep a few more values in flight.
constexpr int blocks_per_cu(bool quant, int group) { return quant && group < 128 ? 3 : 4; }

struct Lds {
  uint16_t* scales;
  uint8_t* zeros;
  float* sums;
};

// One tile: up to 16 rows of expert e by kCols columns. The wavefronts take
// consecutive parts of the steps of k and add their sums in LDS.
template <int DT, bool QUANT, int G, bool ZEROS>
__device__ __forceinline__ void run_tile(const Lds& lds, int32_t H, int64_t N, int e,
                                         int64_t row0, int32_t rows, int64_t n0, const char* x,
                                         const char* w, const uint16_t* scales,
                                         const uint8_t* zeros, void* out) {
  using T = Tile<DT, QUANT, G, ZEROS>;
  constexpr int kStep = T::kStep;
  const int lane = lane_id(), i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t w_row = QUANT ? H / 2 : H * 2;
  const int32_t cols = (int32_t)(N - n0 < kCols ? N - n0 : kCols);
  Source src;
  src.w = w + ((int64_t)e * N + n0) * w_row;
  src.x = x + row0 * H * 2;
  static_for<kNF>([&](auto j) {
    const int32_t n = j * 16 + i16;
    src.w_off[j] = (uint32_t)(n < cols ? n : cols - 1) * w_row;
  });
  src.x_off = (uint32_t)(i16 < rows ? i16 : rows - 1) * (uint32_t)(H * 2);
  f32x4 acc[kNF];
  static_for<kNF>([&](auto j) { acc[j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
  for (int32_t c0 = 0; c0 < H; c0 += QUANT ? kStageK : H) {
    const int32_t left = H - c0;
    const int32_t span = QUANT && left > kStageK ? kStageK : left;
    const int32_t steps = (span + kStep - 1) / kStep;
    const int32_t per = (steps + kWaves - 1) / kWaves;
    int32_t s0 = wave * per;
    const int32_t s1 = s0 + per < steps ? s0 + per : steps;
    typename T::S a, b;
    if (s0 < s1) T::load(a, src, c0 + s0 * kStep, H);
    if constexpr (QUANT) {
      // the scales of the span, transposed to [group][column]; groups past
      // the end of the row and columns past N are zeros
      const int32_t groups = steps * T::kGroups;
      const int64_t all = H / G, g0 = c0 / G;
      __syncthreads();
      for (int32_t t = threadIdx.x; t < groups * kCols; t += kThreads) {
        const int32_t n = t / groups, g = t - n * groups;
        const bool in = n < cols && g0 + g < all;
        const int64_t at = ((int64_t)e * N + n0 + n) * all + g0 + g;
        lds.scales[g * kCols + n] = in ? scales[at] : 0;
        if constexpr (ZEROS) lds.zeros[g * kCols + n] = in ? zeros[at] : 0;
      }
      __syncthreads();
    }
    auto load = [&](typename T::S& to, int32_t s) {
      T::load(to, src, c0 + (s < s1 ? s : s1 - 1) * kStep, H);
    };
    auto multiply = [&](typename T::S& from, int32_t s) {
      const int32_t at = s * T::kGroups * kCols;
      T::multiply(from, c0 + s * kStep, H, lds.scales + at, lds.zeros + at, acc);
    };
    // two steps in turn, each loaded while the other is multiplied
    for (; s0 < s1; s0 += 2) {
      load(b, s0 + 1);
      multiply(a, s0);
      load(a, s0 + 2);
      if (s0 + 1 < s1) multiply(b, s0 + 1);
    }
  }
  static_for<kNF>([&](auto j) {
    float* p = lds.sums + (wave * 16 + i16) * kRedRow + j * 16 + (lane >> 4) * 4;
    *reinterpret_cast<f32x4*>(p) = acc[j];
  });
  __syncthreads();
  // 16 rows x 64 columns by 256 threads: four columns of a row each
  const int m = threadIdx.x / 16, n = threadIdx.x % 16 * 4;
  f32x4 sum = *reinterpret_cast<const f32x4*>(lds.sums + m * kRedRow + n);
  static_for<kWaves - 1>([&](auto v) {
    sum += *reinterpret_cast<const f32x4*>(lds.sums + ((v + 1) * 16 + m) * kRedRow + n);
  });
  if (m < rows && n < cols) {
    u32x2 o;
    if constexpr (DT == EP_DTYPE_BF16) {
      o = u32x2{rne_bf16(sum[0]) | (rne_bf16(sum[1]) << 16),
                rne_bf16(sum[2]) | (rne_bf16(sum[3]) << 16)};
    } else {
      o = u32x2{rne_f16(sum[0]) | (rne_f16(sum[1]) << 16),
                rne_f16(sum[2]) | (rne_f16(sum[3]) << 16)};
    }
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + (row0 + m) * N + n0 + n) = o;
  }
  __syncthreads();  // the sums are read before the next tile writes its own
}

template <int DT, bool QUANT, int G, bool ZEROS>
__global__ void __launch_bounds__(kThreads, blocks_per_cu(QUANT, G))
    few_rows_kernel(Dims d, HandleView hv, const void* __restrict__ x,
                    const void* __restrict__ w, const uint16_t* __restrict__ scales,
                    const uint8_t* __restrict__ zeros, void* __restrict__ out, int64_t N,
                    int32_t scale_bytes) {
  extern __shared__ __align__(16) char mem[];
  Lds lds;
  lds.sums = reinterpret_cast<float*>(mem);
  char* p = mem + kWaves * 16 * kRedRow * sizeof(float);
  lds.scales = reinterpret_cast<uint16_t*>(p);
  p += scale_bytes;
  lds.zeros = reinterpret_cast<uint8_t*>(p);
  if (ZEROS) p += scale_bytes / 2;
  int32_t* tile_start = reinterpret_cast<int32_t*>(p);
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t row_tiles =
      list_tiles<kThreads>(hv, d, kRowTile, tile_start, tile_start + d.E + 1);
  const int64_t ct = (N + kCols - 1) / kCols;
  for (int64_t t = blockIdx.x; t < row_tiles * ct; t += gridDim.x) {
    // the row tiles of an expert are neighbours: they share their weights
    const int e = __builtin_amdgcn_readfirstlane(
        expert_of_tile(tile_start, d.E, (int32_t)(t / ct)));
    const int64_t in_e = t - tile_start[e] * ct;
    const int32_t rts = tile_start[e + 1] - tile_start[e];
    const int32_t ni = __builtin_amdgcn_readfirstlane((int32_t)(in_e / rts));
    const int32_t m0 =
        __builtin_amdgcn_readfirstlane((int32_t)(in_e - (int64_t)ni * rts)) * kRowTile;
    const Segment s = segment_of(hv, d, e);
    run_tile<DT, QUANT, G, ZEROS>(lds, (int32_t)d.H, N, e, s.row + m0,
                                  s.rows - m0 < kRowTile ? s.rows - m0 : kRowTile,
                                  (int64_t)ni * kCols, static_cast<const char*>(x),
                                  static_cast<const char*>(w), scales, zeros, out);
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

template <int DT, bool QUANT, int G, bool ZEROS>
hipError_t launch_few_rows(const Dims& d, const HandleView& hv, const void* x, const void* w,
                           const void* scales, const uint8_t* zeros, void* out, int64_t N,
                           int num_cus, hipStream_t stream) {
  const int64_t ct = (N + kCols - 1) / kCols;
  const int64_t routes = d.T * d.K < d.cap ? d.T * d.K : d.cap;
  int64_t blocks = (routes / kRowTile + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * blocks_per_cu(QUANT, G);
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  size_t scale_bytes = 0;
  if (QUANT) {
    const int64_t span = d.H < kStageK ? d.H : kStageK;
    scale_bytes = (size_t)((span + 127) / 128 * 128 / G) * kCols * 2;
  }
  const size_t lds = kWaves * 16 * kRedRow * sizeof(float) +
                     (ZEROS ? scale_bytes + scale_bytes / 2 : scale_bytes) +
                     sizeof(int32_t) * (size_t)(d.E + 1 + kWaves);
  few_rows_kernel<DT, QUANT, G, ZEROS><<<dim3((uint32_t)blocks), dim3(kThreads), lds, stream>>>(
      d, hv, x, w, static_cast<const uint16_t*>(scales), zeros, out, N, (int32_t)scale_bytes);
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
