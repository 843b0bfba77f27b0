// ep_linear.hip -- products grouped by expert with ragged segments: each
// expert's weights applied to the live rows of its segment, and the two
// gradients of that product.
//
//   forward  C[r, n] = sum_h x[r, h] W[e][n, h]      rows r of expert e
//   dgrad    C[r, h] = sum_n g[r, n] W[e][n, h]
//   wgrad    C[n, h] = sum_r g[r, n] x[r, h]         for every expert e
//
// Each is C = A B over one contraction index k. An operand is K-major when k
// is its contiguous axis (x and W forward, g in dgrad), else MN-major (W in
// dgrad, both operands in wgrad).

#include "ep_choice.h"
#include "ep_experts.h"
#include "ep_tiles.h"

namespace epmi {

namespace {

// One fragment of 16 rows (or columns) of an operand for a lane: 16 bytes, 8
// (16-bit types) or 4 (fp32) values of k. The order of k inside a fragment
// is the same for both operands, which is all that the sum needs.
template <int DT>
__device__ __forceinline__ void mma(f32x4& acc, row16_t n, row16_t m) {
  if constexpr (DT != EP_DTYPE_FP32) {
    acc = mma16<DT>(n, m, acc);
  } else {
    static_for<4>([&](auto t) {
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(n[t.value]),
                                                 __uint_as_float(m[t.value]), acc, 0, 0, 0);
    });
  }
}

// Row tiles of an expert whose column tiles run together: with the columns
// dealt after them, the tiles in flight on an XCD share both operands.
constexpr int kGroup = 6;
// Weight-gradient tiles that go to one XCD together: one for each of its CUs.
constexpr int kChunk = 32;

// One block step is a BM x BN tile of C: WM x WN wavefronts, each with every
// WM-th block of 16 rows and BN / WN columns in registers as 16 x 16 blocks.
// Steps of 128 bytes of k go through two LDS buffers. What comes from the L2
// and beyond takes longer than a step, so a buffer's parts (two halves of the
// rows' operand, the columns') are loaded again each as soon as every
// wavefront has read it out, and waited for a step and a half later: two
// barriers a step, neither of which waits for all loads. Waiting for a whole
// buffer once a step ran at 1353 TFLOP/s on operands of zeros and 1225 on
// random ones against 1535 and 1274 (bf16, 32768 rows of 8 experts, 14336
// inputs, 4096 outputs; a library product of that size 1920 and 1570). The
// clock falls with the operands' bits: on random ones power is the bound.
// Eight wavefronts for the large tile, two a SIMD, so that one's products
// cover the other's LDS reads and barriers; four with twice the columns each
// read a third less from LDS but ran at 1162.
// ONCE: B is expected to be read by one tile alone (a single row tile an
// expert) and passes by the caches; in the weight gradient, C does.
template <int DT, int P, int BM, int BN, int WM, int WN, bool ONCE>
__global__ void __launch_bounds__(WM* WN* kWave)
    grouped_product_kernel(Dims d, HandleView hv, const void* __restrict__ a,
                           const void* __restrict__ b, void* __restrict__ c, int64_t N) {
  // the rows' operand in two halves, the columns' whole
  using A = Operand<DT, P != kWeightGrad, BM / 2, WM>;
  using B = Operand<DT, P == kForward, BN, 1>;
  constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  constexpr int kStage = 2 * A::kBytes + B::kBytes;
  constexpr bool kOnceB = ONCE && P != kWeightGrad, kOnceC = ONCE && P == kWeightGrad;
  constexpr int AL = A::kLoads / kWaves, BL = B::kLoads / kWaves;
  static_assert(AL * kWaves == A::kLoads && BL * kWaves == B::kLoads, "whole loads");
  extern __shared__ __align__(1024) char lds[];
  int32_t* tile_start = reinterpret_cast<int32_t*>(lds + 2 * kStage);
  int32_t* part = tile_start + d.E + 1;

  const int32_t my_rows = rows_of_thread(hv, d);
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t H = d.H;
  const int64_t cols = P == kForward ? N : H;
  const int32_t ct = (int32_t)((cols + BN - 1) / BN);
  const int32_t nt = (int32_t)((N + BM - 1) / BM);  // wgrad: row tiles of every expert
  int64_t tiles;
  if constexpr (P == kWeightGrad) {
    tiles = (int64_t)d.E * nt * ct;
  } else {
    tiles = (int64_t)list_tiles<kThreads>(hv, d, BM, my_rows, tile_start, part) * ct;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int lane = lane_id();
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_char*)lds;
  using std::integral_constant;
  // where this wavefront's fragments lie
  constexpr int kAAt = A::addresses(MF / 2), kBAt = B::addresses(NF);
  uint32_t a_at[kAAt], b_at[kBAt];
  static_for<kAAt>([&](auto i) { a_at[i.value] = lds_base + A::at(wm * 16, i.value); });
  static_for<kBAt>([&](auto i) {
    b_at[i.value] = lds_base + 2 * A::kBytes + B::at(wn * (BN / WN), i.value);
  });
  // Blocks are dealt round-robin to the XCDs: chunks of consecutive tiles go
  // to one XCD each in turn. A grid of fewer blocks than tiles (not wgrad)
  // makes a chunk of what an XCD works on at once.
  const int64_t slots = P == kWeightGrad ? kChunk : gridDim.x / kRunXcds;
  const int64_t xcd = blockIdx.x % kRunXcds, slot = blockIdx.x / kRunXcds;
  int64_t t = ((slot / slots) * kRunXcds + xcd) * slots + slot % slots;
  if constexpr (P == kWeightGrad) t += (int64_t)blockIdx.y * gridDim.x;
  for (; t < tiles; t += P == kWeightGrad ? tiles : (int64_t)gridDim.x) {
    // tile t: expert e, row tile mi, column tile ni
    int e;
    int64_t first;
    int32_t rts;
    if constexpr (P == kWeightGrad) {
      e = (int)(t / ((int64_t)nt * ct));
      first = (int64_t)e * nt * ct;
      rts = nt;
    } else {
      e = expert_of_tile(tile_start, d.E, (int32_t)(t / ct));
      e = __builtin_amdgcn_readfirstlane(e);
      first = (int64_t)tile_start[e] * ct;
      rts = tile_start[e + 1] - tile_start[e];
    }
    const int64_t in_e = t - first;
    const int32_t group = (int32_t)(in_e / ((int64_t)kGroup * ct));
    const int32_t in_g = (int32_t)(in_e - (int64_t)group * kGroup * ct);
    const int32_t gm = rts - group * kGroup < kGroup ? rts - group * kGroup : kGroup;
    const int32_t mi = __builtin_amdgcn_readfirstlane(group * kGroup + in_g % gm);
    const int64_t n0 = __builtin_amdgcn_readfirstlane((in_g / gm) * BN);
    const Segment s = segment_of(hv, d, e);
    const int64_t M = P == kWeightGrad ? N : s.rows;
    // Rows are shared out evenly over a segment's tiles, in blocks of 16: tiles
    // that start together then stay together, and find each other's operands in
    // the L2.
    const int32_t height = (int32_t)(((M + rts - 1) / rts + 15) / 16 * 16);
    const int64_t m0 = (int64_t)mi * height;
    const int32_t depth = (int32_t)(P == kForward ? H : (P == kRowGrad ? N : s.rows));
    const int32_t mrows = (int32_t)(M - m0 < height ? M - m0 : height);
    const int32_t ncols = (int32_t)(cols - n0 < BN ? cols - n0 : BN);
    constexpr int kSize = A::kSize;

    // sources of the two operands and their row (line) strides in bytes
    const uint32_t a_stride = (uint32_t)((P == kForward ? H : N) * kSize);
    const uint32_t b_stride = (uint32_t)(H * kSize);
    const char* a_src = static_cast<const char*>(a);
    const char* b_src = static_cast<const char*>(b);
    if constexpr (P == kWeightGrad) {
      a_src += s.row * a_stride + m0 * kSize;
      b_src += s.row * b_stride + n0 * kSize;
    } else {
      a_src += (s.row + m0) * a_stride;
      b_src += (int64_t)e * N * b_stride + (P == kForward ? n0 * b_stride : n0 * kSize);
    }
    const int32_t steps = pieces(depth, A::kDepth);
    uint32_t a_off[2][AL], b_off[BL];
    static_for<AL>([&](auto i) {
      static_for<2>([&](auto h) {
        a_off[h][i] = A::source(wave * AL + i, a_stride, mrows - h * (BM / 2));
      });
    });
    static_for<BL>([&](auto i) { b_off[i] = B::source(wave * BL + i, b_stride, ncols); });

    // A part (0, 1: the halves of A, 2: B) of step k: its source and its place
    // in LDS. A step past the last has an empty buffer: its loads put zeros into
    // LDS.
    struct Part {
      row16_t buffer;
      uint32_t to;
    };
    auto part_of = [&](auto part, int k) {
      constexpr bool kRows = part.value < 2;
      constexpr bool kMajor = kRows ? P != kWeightGrad : P == kForward;
      constexpr int n = kRows ? AL : BL;
      constexpr int kSkip = kRows ? part.value * (BM / 2) : 0;  // rows before the part
      uint32_t* off = kRows ? a_off[part.value & 1] : b_off;
      const uint32_t k0 = (uint32_t)k * A::kDepth;
      const int32_t left = rest_after(depth, k0);
      const uint32_t stride = kRows ? a_stride : b_stride;
      const int32_t held = (kRows ? mrows : ncols) - kSkip;   // rows or columns of the part
      const char* src = kRows ? a_src : b_src;
      Part p;
      if constexpr (kMajor) {
        if (left > 0 && left < A::kDepth) {
          // the last step: chunks past the end of a row are taken out
          const uint32_t out = A::chunk_k() < left ? 0 : kOutside;
          static_for<n>([&](auto i) { off[i] |= out; });
        }
        const uint32_t byte0 = k0 * kSize;
        p.buffer = buffer_of(src + (int64_t)kSkip * stride + byte0,
                             left > 0 && held > 0 ? (uint32_t)held * stride - byte0 : 0);
      } else {
        const uint32_t lines = left < 0 ? 0 : left < A::kDepth ? left : A::kDepth;
        p.buffer = buffer_of(src + (int64_t)k0 * stride + kSkip * kSize,
                             lines > 0 && held > 0 ? lines * stride - kSkip * kSize : 0);
      }
      p.to = __builtin_amdgcn_readfirstlane(lds_base + (k & 1) * kStage +
                                            part.value * A::kBytes + wave * n * 1024);
      return p;
    };
    auto load_at = [&](auto part, const Part& p, auto i) {
      load_to_lds<(part.value == 2 && kOnceB), i.value * 1024>(
          p.buffer, part.value == 2 ? b_off[i.value] : a_off[part.value & 1][i.value], p.to);
    };
    auto load_part = [&](auto part, int k) {
      const Part p = part_of(part, k);
      static_for<part.value == 2 ? BL : AL>([&](auto i) { load_at(part, p, i); });
    };

    f32x4 acc[MF][NF];
    static_for<MF>([&](auto i) {
      static_for<NF>([&](auto j) { acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    });
    // Fragments: the columns' of both halves of k, the rows' in a ring of four,
    // read kAhead groups of products ahead. Group g of a step is row fragment
    // g / 2 with half g % 2 of k, times every column fragment.
    constexpr int kAhead = MF >= 4 ? 3 : 1;
    constexpr int kGroups = 2 * MF, kMid = MF - kAhead, kEnd = kGroups - kAhead;
    row16_t nf[2][NF], mf[4];
    auto read_n = [&](int k, auto half, auto f) {
      const uint32_t base = b_at[P == kForward ? half.value : f.value] + (k & 1) * kStage;
      nf[half.value][f.value] = B::template read<f.value, half.value>(base);
    };
    auto read_m = [&](int k, auto g) {
      constexpr int half = g.value % 2, f = g.value / 2 % (MF / 2), part = g.value / MF;
      const uint32_t base =
          a_at[P != kWeightGrad ? half : f] + (k & 1) * kStage + part * A::kBytes;
      mf[g.value % 4] = A::template read<f, half>(base);
    };
    constexpr integral_constant<int, 0> i0{};
    constexpr integral_constant<int, 1> i1{};
    constexpr integral_constant<int, 2> i2{};
    // One load every EVERY products of a stretch.
    auto spread = [&](auto part, const Part& p, auto slot, auto first, auto every) {
      constexpr int at = slot.value - first.value * every.value;
      constexpr int n = part.value == 2 ? BL : AL;
      if constexpr (at >= 0 && at % every.value == 0 && at / every.value < n)
        load_at(part, p, integral_constant<int, at / every.value>{});
    };
    // Step k. Two syncs; what is read out at one makes room for loads that are
    // waited for a step and a half later:
    //   mid  A's first half of k and B of k are read out, A's second half has landed
    //   end  A's second half of k is read out, A's first and B of k + 1 have landed
    // The loads are A0 and B of k + 2 at the mid, A1 of k + 2 at the end: at either
    // sync all but the 2 AL + BL youngest have to have landed.
    // Only the first `live` row fragments are multiplied; 0: loads and syncs alone.
    auto step = [&](auto live, int k) {
      Part p0, p1, p2;
      static_for<kGroups>([&](auto g) {
        if constexpr (g.value == kMid) {
          sync_loads<2 * AL + BL>();
          p0 = part_of(i0, k + 2);
          p2 = part_of(i2, k + 2);
        }
        if constexpr (g.value == kEnd) {
          sync_loads<2 * AL + BL>();
          p1 = part_of(i1, k + 2);
        }
        if constexpr (live.value > 0) {
          constexpr int kMidEvery = (kEnd - kMid) * NF / (AL + BL);
          constexpr int kEndEvery = kAhead * NF / AL;
          static_assert(kMidEvery >= 1 && kEndEvery >= 1, "a product for every load");
          constexpr int ahead = (g.value + kAhead) % kGroups;
          if constexpr (ahead / 2 < live.value)
            read_m(g.value + kAhead < kGroups ? k : k + 1, integral_constant<int, ahead>{});
          static_for<NF>([&](auto u) {
            // a set of column fragments is read anew as soon as its last use is past
            if constexpr (g.value == 0) read_n(k, i1, u);
            if constexpr (g.value == kGroups - 1) read_n(k + 1, i0, u);
            if constexpr (g.value >= kMid && g.value < kEnd) {
              constexpr integral_constant<int, (g.value - kMid) * NF + u.value> slot{};
              constexpr integral_constant<int, kMidEvery> every{};
              spread(i0, p0, slot, i0, every);
              spread(i2, p2, slot, integral_constant<int, AL>{}, every);
            }
            if constexpr (g.value >= kEnd) {
              constexpr integral_constant<int, (g.value - kEnd) * NF + u.value> slot{};
              spread(i1, p1, slot, i0, integral_constant<int, kEndEvery>{});
            }
            if constexpr (g.value / 2 < live.value) {
              mma<DT>(acc[g.value / 2][u.value], nf[g.value % 2][u.value], mf[g.value % 4]);
            }
            __builtin_amdgcn_sched_barrier(0);
          });
        } else if constexpr (g.value == kMid) {
          load_part(i0, k + 2);
          load_part(i2, k + 2);
        } else if constexpr (g.value == kEnd) {
          load_part(i1, k + 2);
        }
      });
    };
    auto all_steps = [&](auto live) {
      static_for<2>([&](auto k) {
        load_part(i0, k);
        load_part(i2, k);
        load_part(i1, k);
      });
      sync_loads<2 * AL + BL>();
      if constexpr (live.value > 0) {
        static_for<NF>([&](auto f) { read_n(0, i0, f); });
        static_for<kAhead>([&](auto g) { read_m(0, g); });
      }
      for (int k = 0; k < steps; ++k) step(live, k);
      sync_loads<0>();  // no load is left in flight, and LDS is free again
    };
    const bool busy = wm * 16 < mrows && wn * (BN / WN) < ncols;
    // Power bounds the large tile on ordinary operands, so one whose rows leave
    // fragments empty (row segments end anywhere) leaves their products out, in
    // steps of a quarter down to a half: with the rows shared out evenly, 256 rows
    // an expert on average 306 -> 280 us (row gradient), a share of 32 experts
    // of 1027 rows 1712 -> 1666.
    constexpr bool kTrim = BM == 256 && P != kWeightGrad;
    const int fragments = (mrows + 16 * WM - 1) / (16 * WM);
    if (steps > 0) {
      if (!busy) {
        all_steps(i0);
      } else if (kTrim && fragments <= MF / 2) {
        all_steps(integral_constant<int, kTrim ? MF / 2 : MF>{});
      } else if (kTrim && fragments <= MF * 3 / 4) {
        all_steps(integral_constant<int, kTrim ? MF * 3 / 4 : MF>{});
      } else {
        all_steps(integral_constant<int, MF>{});
      }
    }
    // a lane holds four consecutive columns of one row of each 16 x 16 block
    if (busy) {
      static_for<MF>([&](auto i) {
        const int32_t m = (i * WM + wm) * 16 + (lane & 15);
        const int64_t r = P == kWeightGrad ? (int64_t)e * N + m0 + m : s.row + m0 + m;
        char* to = static_cast<char*>(c) + (r * cols + n0) * kSize;
        if constexpr (DT == EP_DTYPE_FP32) {
          static_for<NF>([&](auto j) {
            const int32_t n = wn * (BN / WN) + j * 16 + (lane >> 4) * 4;
            const f32x4 v = acc[i][j];
            if (m < mrows && n < ncols)
              *reinterpret_cast<row16_t*>(to + n * kSize) =
                  row16_t{canon_f32(v[0]), canon_f32(v[1]), canon_f32(v[2]), canon_f32(v[3])};
          });
        } else {
          static_for<NF / 2>([&](auto j) {
            const row16_t v = join_blocks(round4<DT>(acc[i][2 * j]), round4<DT>(acc[i][2 * j + 1]));
            const int32_t n = wn * (BN / WN) + j * 32 + (lane >> 4) * 8;
            if (m < mrows && n < ncols) {
              row16_t* at = reinterpret_cast<row16_t*>(to + n * kSize);
              if constexpr (kOnceC) {
                store_stream16(at, v);
              } else {
                *at = v;
              }
            }
          });
        }
      });
    }
  }
  if constexpr (P != kWeightGrad) {
    write_zero_rows(hh, hv, d, c, cols * A::kSize / 16);
  }
}

template <int DT, int P, int BM, int BN, int WM, int WN, bool ONCE = false>
hipError_t launch_tiles(const Dims& d, const HandleView& hv, const void* a, const void* b,
                        void* c, int64_t N, int num_cus, int per_cu, hipStream_t stream) {
  auto* kernel = grouped_product_kernel<DT, P, BM, BN, WM, WN, ONCE>;
  const int64_t cols = P == kForward ? N : d.H;
  const int64_t ct = (cols + BN - 1) / BN;
  // the most row tiles that the routing may need: those of all rows, and one part
  // tile an expert
  const int64_t routes = most_rows(d);
  int64_t blocks;
  if (P == kWeightGrad) {
    blocks = (int64_t)d.E * ((N + BM - 1) / BM) * ct;
  } else {
    blocks = (routes / BM + (d.E < routes ? d.E : routes)) * ct;
    const int64_t most = (int64_t)num_cus * per_cu;
    if (blocks > most) blocks = most;
  }
  const int64_t unit = P == kWeightGrad ? kRunXcds * kChunk : kRunXcds;
  blocks = (blocks + unit - 1) / unit * unit;
  if (blocks < unit) blocks = unit;
  // A grid has less than 2^32 threads in one direction: what is past them (2048
  // experts of 8 x 2^20 weights) lies in the other.
  const int64_t most = (int64_t)0xFFFFFFFF / (WM * WN * kWave) / unit * unit;
  const int64_t deep = (blocks + most - 1) / most;
  if (deep > 1) blocks = most;
  const size_t lds = 2 * (size_t)(BM + BN) * 128 + sizeof(int32_t) * (size_t)(d.E + 1 + 16);
  kernel<<<dim3((uint32_t)blocks, (uint32_t)deep), dim3(WM * WN * kWave), lds, stream>>>(
      d, hv, a, b, c, N);
  return hipGetLastError();
}

template <int P>
hipError_t launch_product(const Dims& d, const HandleView& hv, const void* a, const void* b,
                          void* c, int64_t N, int num_cus, hipStream_t stream) {
  const Kernel kernel = kernel_of((Product)P, d, N, num_cus);
  return with_payload(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    constexpr bool kWeights = P == kWeightGrad;
    if constexpr (DT != EP_DTYPE_FP32) {
      switch (kernel) {
        case Kernel::kFewRows:
          return launch_grouped_few(d, hv, a, b, c, N, num_cus, stream);
        case Kernel::kTile256:
          return launch_tiles<DT, P, 256, 256, 2, 4>(d, hv, a, b, c, N, num_cus, 1, stream);
        case Kernel::kTile256Once:
          return launch_tiles<DT, P, 256, 256, 2, 4, kWeights>(d, hv, a, b, c, N, num_cus, 1,
                                                               stream);
        case Kernel::kTile128Once:
          return launch_tiles<DT, P, 128, 128, 2, 2, !kWeights>(d, hv, a, b, c, N, num_cus, 2,
                                                                stream);
        default: break;
      }
    }
    if (kernel == Kernel::kTile64)
      return launch_tiles<DT, P, 64, 64, 2, 2>(d, hv, a, b, c, N, num_cus, 4, stream);
    return launch_tiles<DT, P, 128, 128, 2, 2>(d, hv, a, b, c, N, num_cus, 2, stream);
  });
}

}  // namespace

hipError_t launch_grouped_linear(const Dims& d, const HandleView& hv, const void* x,
                                 const void* weight, void* out, int64_t N, int num_cus,
                                 hipStream_t stream) {
  return launch_product<kForward>(d, hv, x, weight, out, N, num_cus, stream);
}

hipError_t launch_grouped_linear_bwd(const Dims& d, const HandleView& hv, const void* grad,
                                     const void* x, const void* weight, void* grad_x,
                                     void* grad_weight, int64_t N, int num_cus,
                                     hipStream_t stream) {
  if (grad_x) {
    const hipError_t e =
        launch_product<kRowGrad>(d, hv, grad, weight, grad_x, N, num_cus, stream);
    if (e != hipSuccess) return e;
  }
  if (grad_weight)
    return launch_product<kWeightGrad>(d, hv, grad, x, grad_weight, N, num_cus, stream);
  return hipSuccess;
}

}  // namespace epmi
