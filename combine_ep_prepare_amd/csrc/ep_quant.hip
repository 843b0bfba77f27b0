// ep_quant.hip -- the grouped product with 4-bit weights: each value is
// (q - z) * s with one scale s and one zero point z per group of consecutive
// inputs of an output.

#include "ep_experts.h"

namespace epmi {

namespace {

constexpr int kThreads = 256;

// One output column of one expert per wavefront step: the lanes split the
// inputs, dequantise each weight once and apply it to the segment's rows in
// turn.
template <int DT>
__global__ void __launch_bounds__(kThreads)
    grouped_quant_kernel(Dims d, HandleView hv, const void* __restrict__ x,
                         const uint8_t* __restrict__ q, const void* __restrict__ scales,
                         const uint8_t* __restrict__ zeros, void* __restrict__ out, int64_t N,
                         int32_t G) {
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t H = d.H, groups = H / G;
  const int waves = kThreads / kWave, lane = lane_id();
  for (int64_t i = (int64_t)blockIdx.x * waves + threadIdx.x / kWave; i < d.E * N;
       i += (int64_t)gridDim.x * waves) {
    const Segment s = segment_of(hv, d, (int)(i / N));
    for (int32_t m = 0; m < s.rows; ++m) {
      float acc = 0.f;
      for (int64_t k = 2 * lane; k < H; k += 2 * kWave) {
        const int64_t g = i * groups + k / G;
        const float sc = load_elem<DT>(scales, g);
        const float z = zeros ? (float)zeros[g] : 8.f;
        const uint32_t b = q[(i * H + k) / 2];
        const int64_t at = (s.row + m) * H + k;
        acc = __builtin_fmaf(((float)(b & 15u) - z) * sc, load_elem<DT>(x, at), acc);
        acc = __builtin_fmaf(((float)(b >> 4) - z) * sc, load_elem<DT>(x, at + 1), acc);
      }
      static_for<6>([&](auto b) { acc += __shfl_xor(acc, 1 << b, kWave); });
      if (lane == 0) store_elem<DT>(out, (s.row + m) * N + i % N, acc);
    }
  }
  write_zero_rows(hh, hv, d, out, N * 2 / 16);
}

}  // namespace

hipError_t launch_grouped_quant(const Dims& d, const HandleView& hv, const void* x,
                                const uint8_t* q, const void* scales, const uint8_t* zeros,
                                void* out, int64_t N, int32_t group, int num_cus,
                                hipStream_t stream) {
  const dim3 grid(num_cus * 8), block(kThreads);
  if (d.dtype == EP_DTYPE_FP16) {
    grouped_quant_kernel<EP_DTYPE_FP16>
        <<<grid, block, 0, stream>>>(d, hv, x, q, scales, zeros, out, N, group);
  } else {
    grouped_quant_kernel<EP_DTYPE_BF16>
        <<<grid, block, 0, stream>>>(d, hv, x, q, scales, zeros, out, N, group);
  }
  return hipGetLastError();
}

}  // namespace epmi
