// ep_experts.h -- device helpers of the kernels that work on the expert
// segments of a receive buffer (ep_linear.hip, ep_decode.hip, ep_swiglu.hip):
// the live rows of a segment, the list of row tiles over all segments, and
// the zero rows of an output of any width.
#pragma once

#include "ep_device.h"

namespace epmi {

namespace {

// Pieces of `size` that n is cut into, the last one perhaps a part.
__host__ __device__ constexpr int32_t pieces(int32_t n, int32_t size) {
  return n / size + (n % size != 0 ? 1 : 0);
}

// n - at, where `at` is at most a read-ahead past n: both may lie next to 2^31.
__host__ __device__ constexpr int32_t rest_after(int32_t n, uint32_t at) {
  return (int32_t)((uint32_t)n - at);
}

// The live rows of expert e: its valid routes' rows below the capacity. Pad
// rows and rows dropped past the capacity are no operand of any product.
struct Segment {
  int64_t row;   // first received row
  int32_t rows;  // live rows
};

__device__ __forceinline__ Segment segment_of(const HandleView& hv, const Dims& d, int e) {
  Segment s;
  s.row = hv.offsets[e];
  const int64_t room = d.cap - s.row;
  const int64_t n = hv.counts[e];
  s.rows = (int32_t)(room < 0 ? 0 : (n < room ? n : room));
  return s;
}

// tile_start[e] (LDS, E + 1 entries) = the number of row tiles of bm rows
// before expert e; returns their total. Every thread of the block calls it
// with the live rows of expert threadIdx.x, which it has asked for ahead of
// the handle check (the handle's maps are there whatever they hold); part
// holds one word per wavefront. The barriers inside make the list visible to
// the whole block.
__device__ __forceinline__ int32_t rows_of_thread(const HandleView& hv, const Dims& d) {
  return (int)threadIdx.x < d.E ? segment_of(hv, d, (int)threadIdx.x).rows : 0;
}
template <int THREADS>
__device__ __forceinline__ int32_t list_tiles(const HandleView& hv, const Dims& d, int bm,
                                              int32_t first_rows, int32_t* tile_start,
                                              int32_t* part) {
  constexpr int kWaves = THREADS / kWave;
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  int32_t base = 0;
  for (int e0 = 0; e0 < d.E; e0 += THREADS) {
    const int e = e0 + (int)threadIdx.x;
    const int32_t rows = e0 == 0 ? first_rows : e < d.E ? segment_of(hv, d, e).rows : 0;
    const int32_t tiles = pieces(rows, bm);
    int32_t sum = tiles;
    static_for<6>([&](auto i) {
      const int32_t below = __shfl_up(sum, 1u << i, kWave);
      if (lane >= (1 << i)) sum += below;
    });
    if (lane == kWave - 1) part[wave] = sum;
    __syncthreads();
    int32_t before = base, all = 0;
    static_for<kWaves>([&](auto w) {
      const int32_t p = part[w];
      if (w < wave) before += p;
      all += p;
    });
    if (e < d.E) tile_start[e] = before + sum - tiles;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) tile_start[d.E] = base;
  __syncthreads();
  return base;
}

// The expert that holds tile t: the last e with tile_start[e] <= t.
__device__ __forceinline__ int expert_of_tile(const int32_t* tile_start, int E, int32_t t) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= t) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// Writes the zero rows (pads, tail) of an output of `vecs` 16-byte vectors a
// row: one row per wavefront, dealt over the whole grid.
__device__ __forceinline__ void write_zero_rows(const HandleHeader& hh, const HandleView& hv,
                                                const Dims& d, void* out, int64_t vecs) {
  const ZeroRows z = zero_rows_of(hh, d);
  const int waves = blockDim.x / kWave;
  const int64_t first = (int64_t)blockIdx.x * waves + threadIdx.x / kWave;
  const row16_t zero = {0, 0, 0, 0};
  for (int64_t i = first; i < z.n; i += (int64_t)gridDim.x * waves) {
    row16_t* p = static_cast<row16_t*>(out) + zero_row(z, hv.pad_rows, i) * vecs;
    for (int64_t v = lane_id(); v < vecs; v += kWave) store_stream16(p + v, zero);
  }
}

}  // namespace

// f(std::integral_constant<int, DT>) for the payload type dt.
template <typename F>
inline hipError_t with_payload(int dt, F&& f) {
  switch (dt) {
    case EP_DTYPE_FP16: return f(std::integral_constant<int, EP_DTYPE_FP16>{});
    case EP_DTYPE_FP32: return f(std::integral_constant<int, EP_DTYPE_FP32>{});
    default: return f(std::integral_constant<int, EP_DTYPE_BF16>{});
  }
}

}  // namespace epmi
