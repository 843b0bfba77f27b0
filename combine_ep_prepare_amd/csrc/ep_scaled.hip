// ep_scaled.hip -- products grouped by expert with both operands in 8 bits: e4m3
// values, a scale for every 128 inputs of a row of x and one for every 128 x 128
// weights,
//
//   out[r, n] = sum over blocks b of x_scale[r, b] w_scale[e][n / 128][b] *
//               sum over h in b of x[r, h] W[e][n, h].
//
// The inner sum is one matrix instruction of 16 x 16 x 128 that starts at zero (with
// few rows four of 16-bit operands), the outer one fp32 multiply-adds.

#include "ep_choice.h"
#include "ep_gate.h"
#include "ep_lines.h"
#include "ep_tiles.h"

namespace epmi {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A whole block of 128 e4m3 values of k at once: 32 a lane, in two halves. Of each
// eight neighbouring products the instruction cuts off what lies 13 bits below the largest,
// as the 16 x 16 x 32 one of 8-bit operands does: a sum of products of all sizes is off
// by 2^-11 of the largest (measured; by 2^-20 with 16-bit operands). The tiled products
// take it all the same, at twice the 16-bit rate (8 experts of 4096 rows, 14336 x 4096:
// 1640 us, where the product of 16-bit operands takes 3010 and more); the product for
// few rows widens its operands, in the time that the weights' bytes take anyway.
__device__ __forceinline__ f32x4 mma8(row16_t n0, row16_t n1, row16_t m0, row16_t m1) {
  struct Both { row16_t a, b; };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      __builtin_bit_cast(i32x8, Both{n0, n1}), __builtin_bit_cast(i32x8, Both{m0, m1}), zero, 0,
      0, 0, 0, 0, 0);
}

// A lane's sums in two neighbouring blocks of 16 columns, four each, rounded and
// traded for eight side by side (join_blocks). Rounded in whole numbers, as a NaN
// wants it, the large tile's sums took 4096 cycles of the 100000 of a tile of 32
// steps; see pack().
template <int DT>
__device__ __forceinline__ row16_t round_and_join(f32x4 a, f32x4 b) {
  const float o[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  const row16_t r = pack<DT>(o);
  return join_blocks(u32x2{r[0], r[1]}, u32x2{r[2], r[3]});
}

constexpr int kWaves = 4;             // wavefronts of a block: they split k
constexpr int kThreads = kWaves * kWave;
constexpr int kCols = 64;             // columns of a tile: within a scale's 128
constexpr int kRowTile = 16;          // rows of a tile
constexpr int kBlocksPerCU = 4;

// Up to 16 rows of an expert by kCols columns a block step (see ep_lines.h); bound by
// the weights' bytes, which it reads at 6.9 TB/s (32 tokens by top-8 of 256, 7168 x
// 4096: 694 us). The wavefronts take the steps of k in turn, so that the block reads
// 512 bytes of a column side by side, and add their sums in LDS at the end; by then
// each has the first loads of the block's next tile in flight.
template <int DT>
__global__ void __launch_bounds__(kThreads, kBlocksPerCU)
    few_rows_scaled_kernel(Dims d, HandleView hv, const uint8_t* __restrict__ x,
                           const float* __restrict__ x_scales, const uint8_t* __restrict__ w,
                           const float* __restrict__ w_scales, uint16_t* __restrict__ out,
                           int64_t N) {
  using S = Lines<kScaled, DT, kCols>;
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
  const int32_t KB = pieces(H, kScaleBlock), SX = (int32_t)EP_SCALE_COLUMNS(H);
  const int32_t NB = (int32_t)((N + kScaleBlock - 1) / kScaleBlock);
  const int lane = lane_id(), i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  char* lds = mem + wave * S::kLds;

  struct Place {
    typename S::Source src;
    int64_t out;   // first row and column of the tile in `out`
    int32_t rows, cols;
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
    const int64_t n0 = (int64_t)ni * kCols;
    Place p;
    p.rows = s.rows - m0 < kRowTile ? s.rows - m0 : kRowTile;
    p.cols = (int32_t)(N - n0 < kCols ? N - n0 : kCols);
    p.out = (s.row + m0) * N + n0;
    const int64_t row = s.row + m0 + (i16 < p.rows ? i16 : p.rows - 1);
    p.src.w[0] = reinterpret_cast<const char*>(w) + ((int64_t)e * N + n0) * H;
    p.src.cols[0] = p.cols < kCols / 2 ? p.cols : kCols / 2;
    p.src.cols[1] = p.cols - p.src.cols[0];
    p.src.w[1] = p.src.w[0] + (p.src.cols[1] > 0 ? (int64_t)(kCols / 2) * H : 0);
    p.src.x = reinterpret_cast<const char*>(x) + row * H;
    p.src.x_scales = x_scales + row * SX;
    p.src.w_scales[0] = w_scales + ((int64_t)e * NB + n0 / kScaleBlock) * KB;
    return p;
  };
  S s;
  Place next;
  if ((int64_t)blockIdx.x < tiles) {
    next = place(blockIdx.x);
    s.first(next.src, wave, H);
  }
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Place cur = next;
    f32x4 acc[S::kNF];
    static_for<S::kNF>([&](auto j) { acc[j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    s.steps(lds, cur.src, wave, kWaves, H, acc);
    if (t + gridDim.x < tiles) {
      next = place(t + gridDim.x);
      s.first(next.src, wave, H);
    }
    S::put_sums(lds, acc);
    __syncthreads();
    // four columns of a row a thread
    const int m = threadIdx.x / (kCols / 4), n = threadIdx.x % (kCols / 4) * 4;
    if (m < cur.rows && n < cur.cols)
      *reinterpret_cast<u32x2*>(out + cur.out + m * N + n) =
          round4<DT>(S::template sum_of<kWaves>(mem, m, n));
    __syncthreads();  // the sums are read before the next tile's weights
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

// Row tiles of an expert whose column tiles run together: with the columns
// dealt after them, the tiles in flight on an XCD share both operands. 8 experts of
// 4096 rows, 4096 x 28672: 3495 us, against 3545 with 8, 3600 with 6 and 3635 with 12
// (14336 x 4096: 1700, 1710, 1787, 1790; a share of 32 experts of 1024 rows, 7168 x
// 4096, within 2%).
constexpr int kGroup = 4;

// Where tile t lies: t counts an expert's tiles in groups of kGroup row tiles, each
// column of a group after the other, and rows are shared out evenly over a segment's
// row tiles, in blocks of 16.
struct TilePlace {
  int e;
  int32_t rows, cols;    // of the tile
  int64_t row, n0;       // the first of them
};
template <int BN>
__device__ __forceinline__ TilePlace place_of(const HandleView& hv, const Dims& d,
                                              const int32_t* tile_start, int64_t t, int32_t ct,
                                              int64_t N) {
  TilePlace p;
  p.e = __builtin_amdgcn_readfirstlane(expert_of_tile(tile_start, d.E, (int32_t)(t / ct)));
  const int32_t rts = tile_start[p.e + 1] - tile_start[p.e];
  const int64_t in_e = t - (int64_t)tile_start[p.e] * ct;
  const int32_t group = (int32_t)(in_e / ((int64_t)kGroup * ct));
  const int32_t in_g = (int32_t)(in_e - (int64_t)group * kGroup * ct);
  const int32_t gm = rts - group * kGroup < kGroup ? rts - group * kGroup : kGroup;
  const int32_t mi = __builtin_amdgcn_readfirstlane(group * kGroup + in_g % gm);
  p.n0 = __builtin_amdgcn_readfirstlane((in_g / gm) * BN);
  const Segment s = segment_of(hv, d, p.e);
  const int32_t height = (int32_t)((((int64_t)s.rows + rts - 1) / rts + 15) / 16 * 16);
  const int64_t m0 = (int64_t)mi * height;
  p.rows = (int32_t)(s.rows - m0 < height ? s.rows - m0 : height);
  p.cols = (int32_t)(N - p.n0 < BN ? N - p.n0 : BN);
  p.row = s.row + m0;
  return p;
}

// Many rows: the tiled product of ep_linear.hip with steps of 128 values of k, one
// block of scales each. WM x WN wavefronts hold every WM-th block of 16 rows and
// BN / WN columns of a BM x BN tile. A step's parts (two halves of the rows, the
// columns) are loaded again as soon as every wavefront has read them out, and
// waited for a step and a half later.
//
// A matrix instruction gives a whole block's sum of a 16 x 16 part, which is scaled
// and added to the accumulators (four multiply-adds) while the next row fragment's
// instructions run. A row's scales come through LDS too, four steps' at a time, 16
// bytes a row; the columns' one of a step is the same for a wavefront, whose columns
// lie in one block.
//
// 8 experts of 4096 rows: 2200 TFLOP/s at 4096 x 28672, 2270 at 14336 x 4096 (a
// library product of 8-bit operands without scales 3000). The clock falls to 1.6 GHz
// on random operands (2650 TFLOP/s on zeros), and the matrix units are busy 53% of its
// cycles: power is not all of it. Two wavefronts a SIMD leave them idle around the
// syncs, and of seven vector instructions a matrix product four are the multiply-adds
// (2350 TFLOP/s without) and two to three work out offsets and buffers of the next
// loads anew each step, for an end that the last step alone has. More than 256 registers a
// wavefront would let a larger part read less from LDS, but only instructions of the
// matrix unit reach the second half of the file, and the sums need others. 32 x 32 x
// 64 instructions, whose 16 sums a lane spill, ran at 1970.
template <int DT, int BM, int BN, int WM, int WN, bool ONCE>
__global__ void __launch_bounds__(WM* WN* kWave)
    scaled_product_kernel(Dims d, HandleView hv, const uint8_t* __restrict__ x,
                          const float* __restrict__ x_scales, const uint8_t* __restrict__ w,
                          const float* __restrict__ w_scales, uint16_t* __restrict__ out,
                          int64_t N) {
  using A = Operand<kBytes8, true, BM / 2, WM>;
  using B = Operand<kBytes8, true, BN, 1>;
  constexpr int kTileWaves = WM * WN;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  constexpr int kStage = 2 * A::kBytes + B::kBytes;
  constexpr int AL = A::kLoads / kTileWaves, BL = B::kLoads / kTileWaves;
  static_assert(AL * kTileWaves == A::kLoads && BL * kTileWaves == B::kLoads, "whole loads");
  static_assert(BN / WN <= kScaleBlock && MF % 2 == 0, "one column scale, two halves");
  // the row scales of four steps: a wavefront loads 64 rows from its share of them
  // on, the same values that the next ones load
  constexpr int kShare = BM / kTileWaves, kScaleBytes = (BM + 64 - kShare) * 16;
  extern __shared__ __align__(1024) char lds[];
  int32_t* tile_start = reinterpret_cast<int32_t*>(lds + 2 * kStage + 2 * kScaleBytes);

  const int32_t my_rows = rows_of_thread(hv, d);
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int32_t all_H = (int32_t)d.H;
  const int32_t steps = pieces(all_H, kScaleBlock), SX = (int32_t)EP_SCALE_COLUMNS(all_H);
  const int32_t NB = (int32_t)((N + kScaleBlock - 1) / kScaleBlock);
  const int32_t all_ct = (int32_t)((N + BN - 1) / BN);
  // a scalar: as a pair of vector registers it would be spilled over the steps
  const int64_t tiles = (int64_t)__builtin_amdgcn_readfirstlane(list_tiles<kTileWaves * kWave>(
                            hv, d, BM, my_rows, tile_start, tile_start + d.E + 1)) * all_ct;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int lane = lane_id();
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_char*)lds;
  const uint32_t scale_base = lds_base + 2 * kStage;
  using std::integral_constant;
  uint32_t a_at[2], b_at[2];   // of either half of k
  static_for<2>([&](auto i) {
    a_at[i.value] = lds_base + A::at(wm * 16, i.value);
    b_at[i.value] = lds_base + 2 * A::kBytes + B::at(wn * (BN / WN), i.value);
  });
  const uint32_t s_at = scale_base + (wm * 16 + (lane & 15)) * 16;
  // consecutive tiles go to one XCD, as in ep_linear.hip
  const int64_t slots = gridDim.x / kRunXcds;
  const int64_t xcd = blockIdx.x % kRunXcds, slot = blockIdx.x / kRunXcds;
  for (int64_t t = xcd * slots + slot; t < tiles; t += gridDim.x) {
    // What the compiler would work out once and keep over the steps (reciprocals of
    // ct, the lanes' places in a tile) takes registers that the large tile does not
    // have: opaque here and below, it is worked out for each tile.
    int32_t ct = all_ct, H = all_H;
    asm volatile("" : "+s"(ct), "+s"(H));
    const TilePlace at = place_of<BN>(hv, d, tile_start, t, ct, N);
    const int e = at.e;
    const int64_t row = at.row, n0 = at.n0;
    const int32_t mrows = at.rows, ncols = at.cols;
    const char* a_src = reinterpret_cast<const char*>(x) + row * H;
    const char* b_src = reinterpret_cast<const char*>(w) + ((int64_t)e * N + n0) * H;
    uint32_t a_off[2][AL], b_off[BL];
    static_for<AL>([&](auto i) {
      static_for<2>([&](auto h) { a_off[h][i] = A::source(wave * AL + i, (uint32_t)H, 0); });
    });
    static_for<BL>([&](auto i) { b_off[i] = B::source(wave * BL + i, (uint32_t)H, 0); });

    // A part (0, 1: the halves of A, 2: B) of step k: its source and its place
    // in LDS. A step past the last has an empty buffer: its loads put zeros into
    // LDS.
    struct Part {
      row16_t buffer;
      uint32_t to;
    };
    auto part_of = [&](auto part, int k) {
      constexpr bool kRows = part.value < 2;
      constexpr int n = kRows ? AL : BL;
      constexpr int kSkip = kRows ? part.value * (BM / 2) : 0;  // rows before the part
      uint32_t* off = kRows ? a_off[part.value & 1] : b_off;
      const uint32_t k0 = (uint32_t)k * A::kDepth;
      const int32_t left = rest_after(H, k0);
      const int32_t held = (kRows ? mrows : ncols) - kSkip;   // rows or columns of the part
      // in the last step chunks past the end of a row are taken out; without a branch,
      // as below
      const uint32_t gone = A::chunk_k() < left ? 0 : kOutside;
      static_for<n>([&](auto i) { off[i] |= gone; });
      Part p;
      p.buffer = buffer_of((kRows ? a_src : b_src) + (int64_t)kSkip * H + k0,
                           left > 0 && held > 0 ? (uint32_t)held * (uint32_t)H - k0 : 0);
      p.to = __builtin_amdgcn_readfirstlane(lds_base + (k & 1) * kStage +
                                            part.value * A::kBytes + wave * n * 1024);
      return p;
    };
    auto load_at = [&](auto part, const Part& p, auto i) {
      load_to_lds<(part.value == 2 && ONCE), i.value * 1024>(
          p.buffer, part.value == 2 ? b_off[i.value] : a_off[part.value & 1][i.value], p.to);
    };
    auto load_part = [&](auto part, int k) {
      const Part p = part_of(part, k);
      static_for<part.value == 2 ? BL : AL>([&](auto i) { load_at(part, p, i); });
    };
    // the row scales of steps 4 j to 4 j + 3
    const uint32_t s_off = (uint32_t)(wave * kShare + lane) * (uint32_t)(SX * 4);
    auto load_scales = [&](int j) {
      const uint32_t bytes = (uint32_t)mrows * (uint32_t)(SX * 4);
      load_to_lds<false, 0>(buffer_of(x_scales + row * SX, bytes),
                            j * 4 < SX ? s_off + (uint32_t)j * 16 : kOutside,
                            __builtin_amdgcn_readfirstlane(scale_base + (j & 1) * kScaleBytes +
                                                           wave * kShare * 16));
    };
    // the wavefront's column scales
    const int64_t nb = (n0 + wn * (BN / WN)) / kScaleBlock;
    const float* w_scale = w_scales + ((int64_t)e * NB + (nb < NB ? nb : NB - 1)) * steps;

    f32x4 acc[MF][NF];
    static_for<MF>([&](auto i) {
      static_for<NF>([&](auto j) { acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    });
    // Fragments of both halves of k: the columns', and the rows' in a ring, read
    // kAhead row fragments ahead with their scales; and the sums of the last NF
    // products, each of which is added to the accumulators when NF - 1 more have
    // been issued.
    constexpr int kAhead = MF >= 8 ? 2 : 1, kRing = MF >= 4 ? 4 : 2;
    constexpr int kMid = MF / 2 - kAhead, kEnd = MF - kAhead;
    row16_t nf[NF][2], mf[kRing][2];
    float sf[kRing];
    f32x4 sums[NF];
    float by = 0.f;    // scales the next sums to be added
    static_for<NF>([&](auto u) { sums[u] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    auto read_n = [&](int k, auto f) {
      static_for<2>([&](auto h) {
        nf[f.value][h.value] = B::template read<f.value, h.value>(b_at[h.value] + (k & 1) * kStage);
      });
    };
    auto read_m = [&](int k, auto g) {
      constexpr int f = g.value % (MF / 2), part = g.value / (MF / 2);
      static_for<2>([&](auto h) {
        mf[g.value % kRing][h.value] = A::template read<f, h.value>(
            a_at[h.value] + (k & 1) * kStage + part * A::kBytes);
      });
      sf[g.value % kRing] = *reinterpret_cast<const __attribute__((address_space(3))) float*>(
          (const lds_char*)(uintptr_t)(s_at + (k / 4 % 2) * kScaleBytes + (k % 4) * 4 +
                                       g.value * WM * 256));
    };
    constexpr integral_constant<int, 0> i0{};
    constexpr integral_constant<int, 1> i1{};
    constexpr integral_constant<int, 2> i2{};
    auto add_up = [&](auto g, auto u) {   // sums of row fragment g
      static_for<4>([&](auto c) {
        acc[g.value][u.value][c.value] = __builtin_fmaf(
            by, sums[u.value][c.value], acc[g.value][u.value][c.value]);
      });
    };
    // The part's loads of a stretch that issues `all`, of which it holds those from
    // `first` on, over `slots` products.
    auto spread = [&](auto part, const Part& p, auto slot, auto slots, auto all, auto first) {
      constexpr int n = part.value == 2 ? BL : AL;
      static_for<n>([&](auto i) {
        if constexpr ((first.value + i.value) * slots.value / all.value == slot.value)
          load_at(part, p, i);
      });
    };
    // Step k, with two syncs as in ep_linear.hip: at the mid, A's first half of k and
    // B of k are read out and A's second half has landed; at the end, A's second half
    // is read out and the next step's first half and B have landed. Only the first
    // `live` row fragments are multiplied; 0: loads and syncs alone. The scales of
    // four steps are asked for in the first of the four before, ahead of the
    // operands that the syncs count: they have landed a step later.
    auto step = [&](auto live, int k, float w_by) {
      Part p0, p1, p2;
      static_for<MF>([&](auto g) {
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
          constexpr int ahead = (g.value + kAhead) % MF;
          if constexpr (ahead < live.value)
            read_m(g.value + kAhead < MF ? k : k + 1, integral_constant<int, ahead>{});
          static_for<NF>([&](auto u) {
            if constexpr (g.value >= kMid && g.value < kEnd) {
              constexpr integral_constant<int, (g.value - kMid) * NF + u.value> slot{};
              constexpr integral_constant<int, (kEnd - kMid) * NF> slots{};
              constexpr integral_constant<int, AL + BL> all{};
              spread(i0, p0, slot, slots, all, i0);
              spread(i2, p2, slot, slots, all, integral_constant<int, AL>{});
            }
            if constexpr (g.value >= kEnd) {
              constexpr integral_constant<int, (g.value - kEnd) * NF + u.value> slot{};
              spread(i1, p1, slot, integral_constant<int, kAhead * NF>{},
                     integral_constant<int, AL>{}, i0);
            }
            if constexpr (g.value < live.value) {
              sums[u.value] = mma8(nf[u.value][0], nf[u.value][1], mf[g.value % kRing][0],
                                   mf[g.value % kRing][1]);
              if constexpr (u.value < NF - 1) {
                add_up(integral_constant<int, (g.value + live.value - 1) % live.value>{},
                       integral_constant<int, u.value + 1>{});
              } else {
                by = sf[g.value % kRing] * w_by;
                add_up(g, i0);
              }
            }
            // the columns are read anew as soon as their last use is past
            if constexpr (g.value == MF - 1) read_n(k + 1, u);
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
      load_scales(0);
      static_for<2>([&](auto k) {
        load_part(i0, k);
        load_part(i2, k);
        load_part(i1, k);
      });
      sync_loads<2 * AL + BL>();
      if constexpr (live.value > 0) {
        static_for<NF>([&](auto f) { read_n(0, f); });
        static_for<kAhead>([&](auto g) { read_m(0, g); });
      }
      float w_by = w_scale[0];
      for (int k = 0; k < steps; ++k) {
        // Their place's last readers are past the sync at the last step's end. A
        // branch inside the step would let the compiler put the multiply-adds of
        // the products ahead of it behind it, and keep all of their sums till then.
        if (k % 4 == 0) load_scales(k / 4 + 1);
        const float w_next = w_scale[k + 1 < steps ? k + 1 : k];
        step(live, k, w_by);
        w_by = w_next;
      }
      if constexpr (live.value > 0) {
        static_for<NF - 1>([&](auto u) {
          add_up(integral_constant<int, (live.value > 0 ? live.value : 1) - 1>{},
                 integral_constant<int, u.value + 1>{});
        });
      }
      sync_loads<0>();  // no load is left in flight, and LDS is free again
    };
    const bool busy = wm * 16 < mrows && wn * (BN / WN) < ncols;
    // a tile with empty row fragments leaves their products out, in steps of a
    // quarter down to a half
    constexpr bool kTrim = BM == 256;
    const int fragments = (mrows + 16 * WM - 1) / (16 * WM);
    if (!busy) {
      all_steps(i0);
    } else if (kTrim && fragments <= MF / 2) {
      all_steps(integral_constant<int, kTrim ? MF / 2 : MF>{});
    } else if (kTrim && fragments <= MF * 3 / 4) {
      all_steps(integral_constant<int, kTrim ? MF * 3 / 4 : MF>{});
    } else {
      all_steps(integral_constant<int, MF>{});
    }
    // a lane holds four consecutive columns of one row of each 16 x 16 block
    if (busy) {
      int place = lane;
      asm volatile("" : "+v"(place));
      static_for<MF>([&](auto i) {
        const int32_t m = (i * WM + wm) * 16 + (place & 15);
        uint16_t* to = out + (row + m) * N + n0;
        static_for<NF / 2>([&](auto j) {
          const row16_t v = round_and_join<DT>(acc[i][2 * j], acc[i][2 * j + 1]);
          const int32_t n = wn * (BN / WN) + j * 32 + (place >> 4) * 8;
          if (m < mrows && n < ncols) *reinterpret_cast<row16_t*>(to + n) = v;
        });
      });
    }
  }
  // the header again: kept over the loop it would take registers that the large
  // tile does not have
  write_zero_rows(*hv.header, hv, d, out, N * 2 / 16);
}

template <int DT, int BM, int BN, int WM, int WN, bool ONCE>
hipError_t launch_scaled_tiles(const Dims& d, const HandleView& hv, const uint8_t* x,
                               const float* x_scales, const uint8_t* w, const float* w_scales,
                               void* out, int64_t N, int num_cus, int per_cu,
                               hipStream_t stream) {
  constexpr int kTileWaves = WM * WN;
  const int64_t ct = (N + BN - 1) / BN, routes = most_rows(d);
  int64_t blocks = (routes / BM + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * per_cu;
  if (blocks > most) blocks = most;
  blocks = (blocks + kRunXcds - 1) / kRunXcds * kRunXcds;
  if (blocks < kRunXcds) blocks = kRunXcds;
  const size_t lds = 2 * (size_t)(BM + BN) * 128 +
                     2 * (size_t)(BM + 64 - BM / kTileWaves) * 16 +
                     sizeof(int32_t) * (size_t)(d.E + 1 + 16);
  scaled_product_kernel<DT, BM, BN, WM, WN, ONCE>
      <<<dim3((uint32_t)blocks), dim3(kTileWaves * kWave), lds, stream>>>(
          d, hv, x, x_scales, w, w_scales, static_cast<uint16_t*>(out), N);
  return hipGetLastError();
}

// Smaller tiles, where a grid leaves a CU few wavefronts and steps are short: a
// ring of STAGES buffers of a step each, all but one of them asked for ahead, and
// one sync a step: the step's buffer has landed for all wavefronts, and the one that
// the step before read is free again. Layout, scales and results as above.
template <int DT, int BM, int BN, int WM, int WN, int STAGES, bool ONCE>
__global__ void __launch_bounds__(WM* WN* kWave)
    scaled_ring_kernel(Dims d, HandleView hv, const uint8_t* __restrict__ x,
                       const float* __restrict__ x_scales, const uint8_t* __restrict__ w,
                       const float* __restrict__ w_scales, uint16_t* __restrict__ out,
                       int64_t N) {
  using A = Operand<kBytes8, true, BM, WM>;
  using B = Operand<kBytes8, true, BN, 1>;
  constexpr int kTileWaves = WM * WN;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  constexpr int kStage = A::kBytes + B::kBytes;
  constexpr int AL = A::kLoads / kTileWaves, BL = B::kLoads / kTileWaves;
  static_assert(AL * kTileWaves == A::kLoads && BL * kTileWaves == B::kLoads, "whole loads");
  static_assert(BN / WN <= kScaleBlock && NF % 2 == 0, "one column scale, results in pairs");
  static_assert(STAGES <= 4, "two sets of row scales");
  constexpr int kShare = BM / kTileWaves, kScaleBytes = (BM + 64 - kShare) * 16;
  extern __shared__ __align__(1024) char lds[];
  int32_t* tile_start = reinterpret_cast<int32_t*>(lds + STAGES * kStage + 2 * kScaleBytes);

  const int32_t my_rows = rows_of_thread(hv, d);
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int32_t H = (int32_t)d.H;
  const int32_t steps = pieces(H, kScaleBlock), SX = (int32_t)EP_SCALE_COLUMNS(H);
  const int32_t NB = (int32_t)((N + kScaleBlock - 1) / kScaleBlock);
  const int32_t ct = (int32_t)((N + BN - 1) / BN);
  const int64_t tiles = (int64_t)list_tiles<kTileWaves * kWave>(hv, d, BM, my_rows, tile_start,
                                                                tile_start + d.E + 1) * ct;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int lane = lane_id();
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_char*)lds;
  const uint32_t scale_base = lds_base + STAGES * kStage;
  uint32_t a_at[2], b_at[2];   // of either half of k
  static_for<2>([&](auto i) {
    a_at[i.value] = lds_base + A::at(wm * 16, i.value);
    b_at[i.value] = lds_base + A::kBytes + B::at(wn * (BN / WN), i.value);
  });
  const uint32_t s_at = scale_base + (wm * 16 + (lane & 15)) * 16;
  const int64_t slots = gridDim.x / kRunXcds;
  const int64_t xcd = blockIdx.x % kRunXcds, slot = blockIdx.x / kRunXcds;
  for (int64_t t = xcd * slots + slot; t < tiles; t += gridDim.x) {
    const TilePlace at = place_of<BN>(hv, d, tile_start, t, ct, N);
    const int e = at.e;
    const int64_t row = at.row, n0 = at.n0;
    const int32_t mrows = at.rows, ncols = at.cols;
    const char* a_src = reinterpret_cast<const char*>(x) + row * H;
    const char* b_src = reinterpret_cast<const char*>(w) + ((int64_t)e * N + n0) * H;
    const float* s_src = x_scales + row * SX;
    uint32_t a_off[AL], b_off[BL];
    static_for<AL>([&](auto i) { a_off[i] = A::source(wave * AL + i, (uint32_t)H, 0); });
    static_for<BL>([&](auto i) { b_off[i] = B::source(wave * BL + i, (uint32_t)H, 0); });
    const uint32_t s_off = (uint32_t)(wave * kShare + lane) * (uint32_t)(SX * 4);

    // Step k into its buffer, and with every fourth the row scales of four; a step
    // past the last has empty buffers, whose loads put zeros into LDS.
    auto load = [&](int k) {
      const uint32_t k0 = (uint32_t)k * A::kDepth;
      const int32_t left = rest_after(H, k0);
      const uint32_t gone = A::chunk_k() < left ? 0 : kOutside;
      const uint32_t to = lds_base + k % STAGES * kStage;
      if (k % 4 == 0)
        load_to_lds<false, 0>(
            buffer_of(s_src, left > 0 ? (uint32_t)mrows * (uint32_t)(SX * 4) : 0),
            s_off + (uint32_t)k * 4,
            __builtin_amdgcn_readfirstlane(scale_base + k / 4 % 2 * kScaleBytes +
                                           wave * kShare * 16));
      const row16_t ab = buffer_of(a_src + k0, left > 0 ? (uint32_t)mrows * (uint32_t)H - k0 : 0);
      const row16_t bb = buffer_of(b_src + k0, left > 0 ? (uint32_t)ncols * (uint32_t)H - k0 : 0);
      const uint32_t a_to = __builtin_amdgcn_readfirstlane(to + wave * AL * 1024);
      const uint32_t b_to = __builtin_amdgcn_readfirstlane(to + A::kBytes + wave * BL * 1024);
      static_for<AL>([&](auto i) {
        load_to_lds<false, i.value * 1024>(ab, a_off[i] | gone, a_to);
      });
      static_for<BL>([&](auto i) {
        load_to_lds<ONCE, i.value * 1024>(bb, b_off[i] | gone, b_to);
      });
    };
    const int64_t nb = (n0 + wn * (BN / WN)) / kScaleBlock;
    const float* w_scale = w_scales + ((int64_t)e * NB + (nb < NB ? nb : NB - 1)) * steps;

    f32x4 acc[MF][NF];
    static_for<MF>([&](auto i) {
      static_for<NF>([&](auto j) { acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    });
    const bool busy = wm * 16 < mrows && wn * (BN / WN) < ncols;
    static_for<STAGES - 1>([&](auto k) { load(k); });
    float w_by = w_scale[0];
    for (int k = 0; k < steps; ++k) {
      const float w_next = w_scale[k + 1 < steps ? k + 1 : k];
      // the loads of STAGES - 2 steps may be on their way (where one of them has
      // scales too, an older one is waited for that need not be)
      sync_loads<(STAGES - 2) * (AL + BL)>();
      load(k + STAGES - 1);
      if (busy) {
        const uint32_t at = k % STAGES * kStage;
        row16_t nf[NF][2];
        static_for<NF>([&](auto j) {
          static_for<2>([&](auto h) {
            nf[j][h.value] = B::template read<j.value, h.value>(b_at[h.value] + at);
          });
        });
        static_for<MF>([&](auto i) {
          row16_t mf[2];
          static_for<2>([&](auto h) {
            mf[h.value] = A::template read<i.value, h.value>(a_at[h.value] + at);
          });
          const float by =
              w_by * *reinterpret_cast<const __attribute__((address_space(3))) float*>(
                         (const lds_char*)(uintptr_t)(s_at + k / 4 % 2 * kScaleBytes + k % 4 * 4 +
                                                      i.value * WM * 256));
          static_for<NF>([&](auto j) {
            const f32x4 sum = mma8(nf[j][0], nf[j][1], mf[0], mf[1]);
            static_for<4>([&](auto c) {
              acc[i][j][c.value] = __builtin_fmaf(by, sum[c.value], acc[i][j][c.value]);
            });
          });
        });
      }
      w_by = w_next;
    }
    sync_loads<0>();  // no load is left in flight, and LDS is free again
    // a lane holds four consecutive columns of one row of each 16 x 16 block
    if (busy) {
      static_for<MF>([&](auto i) {
        const int32_t m = (i * WM + wm) * 16 + (lane & 15);
        uint16_t* to = out + (row + m) * N + n0;
        static_for<NF / 2>([&](auto j) {
          const row16_t v = round_and_join<DT>(acc[i][2 * j], acc[i][2 * j + 1]);
          const int32_t n = wn * (BN / WN) + j * 32 + (lane >> 4) * 8;
          if (m < mrows && n < ncols) *reinterpret_cast<row16_t*>(to + n) = v;
        });
      });
    }
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

template <int DT, int BM, int BN, int WM, int WN, int STAGES, bool ONCE>
hipError_t launch_scaled_ring(const Dims& d, const HandleView& hv, const uint8_t* x,
                              const float* x_scales, const uint8_t* w, const float* w_scales,
                              void* out, int64_t N, int num_cus, int per_cu, hipStream_t stream) {
  constexpr int kTileWaves = WM * WN;
  const int64_t ct = (N + BN - 1) / BN, routes = most_rows(d);
  int64_t blocks = (routes / BM + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * per_cu;
  if (blocks > most) blocks = most;
  blocks = (blocks + kRunXcds - 1) / kRunXcds * kRunXcds;
  if (blocks < kRunXcds) blocks = kRunXcds;
  const size_t lds = STAGES * (size_t)(BM + BN) * 128 +
                     2 * (size_t)(BM + 64 - BM / kTileWaves) * 16 +
                     sizeof(int32_t) * (size_t)(d.E + 1 + 16);
  scaled_ring_kernel<DT, BM, BN, WM, WN, STAGES, ONCE>
      <<<dim3((uint32_t)blocks), dim3(kTileWaves * kWave), lds, stream>>>(
          d, hv, x, x_scales, w, w_scales, static_cast<uint16_t*>(out), N);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_few_rows(const Dims& d, const HandleView& hv, const uint8_t* x,
                           const float* x_scales, const uint8_t* w, const float* w_scales,
                           void* out, int64_t N, int num_cus, int per_cu, hipStream_t stream) {
  const int64_t ct = (N + kCols - 1) / kCols;
  const int64_t routes = most_rows(d);
  int64_t blocks = (routes / kRowTile + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * per_cu;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  const size_t lds = kWaves * (size_t)Lines<kScaled, DT, kCols>::kLds +
                     sizeof(int32_t) * (size_t)(d.E + 1 + kWaves);
  few_rows_scaled_kernel<DT><<<dim3((uint32_t)blocks), dim3(kThreads), lds, stream>>>(
      d, hv, x, x_scales, w, w_scales, static_cast<uint16_t*>(out), N);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_product(const Dims& d, const HandleView& hv, const uint8_t* x,
                          const float* x_scales, const uint8_t* w, const float* w_scales,
                          void* out, int64_t N, int num_cus, hipStream_t stream) {
  auto go = [&](auto launch, int per_cu) {
    return launch(d, hv, x, x_scales, w, w_scales, out, N, num_cus, per_cu, stream);
  };
  switch (scaled_kernel_of(d, N, num_cus)) {
    case Kernel::kTile256: return go(launch_scaled_tiles<DT, 256, 256, 2, 4, false>, 1);
    case Kernel::kTile256Once: return go(launch_scaled_tiles<DT, 256, 256, 2, 4, true>, 1);
    case Kernel::kTile128: return go(launch_scaled_tiles<DT, 128, 128, 2, 2, false>, 2);
    case Kernel::kTile128Once: return go(launch_scaled_tiles<DT, 128, 128, 2, 2, true>, 2);
    case Kernel::kTile64: return go(launch_scaled_tiles<DT, 64, 64, 2, 2, false>, 4);
    case Kernel::kRing64: return go(launch_scaled_ring<DT, 64, 64, 2, 2, 4, false>, 2);
    case Kernel::kRing128: return go(launch_scaled_ring<DT, 128, 128, 2, 4, 4, false>, 1);
    case Kernel::kRing64x128: return go(launch_scaled_ring<DT, 64, 128, 2, 4, 3, true>, 2);
    case Kernel::kFewRows: break;
  }
  return go(launch_few_rows<DT>, kBlocksPerCU);
}

}  // namespace

hipError_t launch_grouped_scaled(const Dims& d, const HandleView& hv, const uint8_t* x,
                                 const float* x_scales, const uint8_t* w, const float* w_scales,
                                 void* out, int64_t N, int num_cus, hipStream_t stream) {
  if (d.dtype == EP_DTYPE_FP16)
    return launch_product<EP_DTYPE_FP16>(d, hv, x, x_scales, w, w_scales, out, N, num_cus,
                                          stream);
  return launch_product<EP_DTYPE_BF16>(d, hv, x, x_scales, w, w_scales, out, N, num_cus, stream);
}

}  // namespace epmi
