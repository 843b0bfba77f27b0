// ep_scaled.hip -- products grouped by expert with both operands in 8 bits: e4m3
// values, a scale for every 128 inputs of a row of x and one for every 128 x 128
// weights,
//
//   out[r, n] = sum over blocks b of x_scale[r, b] w_scale[e][n / 128][b] *
//               sum over h in b of x[r, h] W[e][n, h].
//
// The inner sum is one matrix instruction of 16 x 16 x 128 that starts at zero,
// the outer one fp32 multiply-adds.

#include "ep_lines.h"

namespace epmi {

namespace {

constexpr int kWaves = 4;             // wavefronts of a block: they split k
constexpr int kThreads = kWaves * kWave;
constexpr int kCols = 64;             // columns of a tile: within a scale's 128
constexpr int kRowTile = 16;          // rows of a tile
constexpr int kBlocksPerCU = 4;

// Up to 16 rows of an expert by kCols columns a block step (see ep_lines.h). The
// wavefronts take the steps of k in turn, so that the block reads 512 bytes of a
// column side by side, and add their sums in LDS at the end; by then each has the
// first loads of the block's next tile in flight.
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
          round_four<DT>(S::template sum_of<kWaves>(mem, m, n));
    __syncthreads();  // the sums are read before the next tile's weights
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

// The most rows that all experts together can have (ep_choice.h).
inline int64_t most_rows(const Dims& d) {
  const int64_t routes = d.T * d.K;
  return routes < d.cap ? routes : d.cap;
}

template <int DT>
hipError_t launch_few_rows(const Dims& d, const HandleView& hv, const uint8_t* x,
                           const float* x_scales, const uint8_t* w, const float* w_scales,
                           void* out, int64_t N, int num_cus, hipStream_t stream) {
  const int64_t ct = (N + kCols - 1) / kCols;
  const int64_t routes = most_rows(d);
  int64_t blocks = (routes / kRowTile + (d.E < routes ? d.E : routes)) * ct;
  const int64_t most = (int64_t)num_cus * kBlocksPerCU;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  const size_t lds = kWaves * (size_t)Lines<kScaled, DT, kCols>::kLds +
                     sizeof(int32_t) * (size_t)(d.E + 1 + kWaves);
  few_rows_scaled_kernel<DT><<<dim3((uint32_t)blocks), dim3(kThreads), lds, stream>>>(
      d, hv, x, x_scales, w, w_scales, static_cast<uint16_t*>(out), N);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_scaled(const Dims& d, const HandleView& hv, const uint8_t* x,
                                 const float* x_scales, const uint8_t* w, const float* w_scales,
                                 void* out, int64_t N, int num_cus, hipStream_t stream) {
  if (d.dtype == EP_DTYPE_FP16)
    return launch_few_rows<EP_DTYPE_FP16>(d, hv, x, x_scales, w, w_scales, out, N, num_cus,
                                          stream);
  return launch_few_rows<EP_DTYPE_BF16>(d, hv, x, x_scales, w, w_scales, out, N, num_cus, stream);
}

}  // namespace epmi
