// ep_swiglu.hip -- the experts' gated activation over a receive buffer,
//   out = silu(gate) * up,  silu(g) = g * s,  s = 1 / (1 + exp(-g)),
// with gate and up the two halves of a row, and its gradient
//   d_up = grad * g * s,  d_gate = grad * up * s * (1 + g * (1 - s)).
// Both are bound by HBM traffic: rows of 3 (forward) or 5 (backward) times
// the hidden size move once. Everything between the loads and the one
// rounding at the store is fp32.

#include "ep_experts.h"

namespace epmi {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerCU = 8;

__device__ __forceinline__ float sigmoid(float g) { return 1.f / (1.f + expf(-g)); }

// A wavefront step is one 1 KiB piece of an output row (or of each half of a
// gradient row). Rows are taken in address order; row_src tells which hold a
// route, the others are zeroed under the layout's pad and tail policies.
template <int DT, bool BWD>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(Dims d, HandleView hv, const row16_t* __restrict__ grad,
                  const row16_t* __restrict__ gate_up, row16_t* __restrict__ out) {
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  using P = Payload<DT>;
  constexpr int N = P::N;
  const int64_t live = hh.total < d.cap ? hh.total : d.cap;
  const int64_t rows = d.zero_tail ? d.cap : live;
  const int64_t V = d.V, pieces = (V + kWave - 1) / kWave;
  const int waves = kThreads / kWave;
  for (int64_t i = (int64_t)blockIdx.x * waves + threadIdx.x / kWave; i < rows * pieces;
       i += (int64_t)gridDim.x * waves) {
    const int64_t r = i / pieces, v = (i - r * pieces) * kWave + lane_id();
    const bool held = r < live && hv.row_src[r] >= 0;
    if (!held && r < live && !d.fill_pads) continue;
    if (v >= V) continue;
    row16_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (held) {
      const row16_t gv = gate_up[r * 2 * V + v], uv = gate_up[r * 2 * V + V + v];
      row16_t dv = {0, 0, 0, 0};
      if constexpr (BWD) dv = grad[r * V + v];
      float o[N], o2[N];
      static_for<N>([&](auto j) {
        const float g = P::template get<j>(gv), u = P::template get<j>(uv);
        const float s = sigmoid(g);
        if constexpr (BWD) {
          const float dd = P::template get<j>(dv);
          o[j] = dd * u * (s * (1.f + g * (1.f - s)));
          o2[j] = dd * (g * s);
        } else {
          o[j] = g * s * u;
        }
      });
      a = P::pack(o);
      if constexpr (BWD) b = P::pack(o2);
    }
    if constexpr (BWD) {
      store_stream16(out + r * 2 * V + v, a);
      store_stream16(out + r * 2 * V + V + v, b);
    } else {
      store_stream16(out + r * V + v, a);
    }
  }
}

}  // namespace

hipError_t launch_swiglu(const Dims& d, const HandleView& hv, bool backward, const void* grad,
                         const void* gate_up, void* out, int num_cus, hipStream_t stream) {
  return with_payload(d.dtype, [&](auto dt) {
    const dim3 grid(num_cus * kBlocksPerCU), block(kThreads);
    const row16_t* g = static_cast<const row16_t*>(grad);
    const row16_t* gu = static_cast<const row16_t*>(gate_up);
    row16_t* o = static_cast<row16_t*>(out);
    if (backward) {
      swiglu_kernel<decltype(dt)::value, true><<<grid, block, 0, stream>>>(d, hv, g, gu, o);
    } else {
      swiglu_kernel<decltype(dt)::value, false><<<grid, block, 0, stream>>>(d, hv, g, gu, o);
    }
    return hipGetLastError();
  });
}

}  // namespace epmi
