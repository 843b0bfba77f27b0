// ep_swiglu.hip -- the experts' gated activation over a receive buffer,
//   out = silu(gate) * up,  silu(g) = g * s,  s = 1 / (1 + exp(-g)),
// with gate and up the two halves of a row, and its gradient
//   d_up = grad * g * s,  d_gate = grad * up * s * (1 + g * (1 - s)).
//
// Both are bound by HBM traffic: 3 (forward) or 5 (backward) times the hidden
// size a row, each value moved once. Everything between the loads and the one
// rounding at the store is fp32. For that bound the arithmetic has to stay
// under about 40 instructions a value of 16 bits, which the library's exp and
// an IEEE quotient alone pass; exp2 and the reciprocal of the hardware (each
// within a unit in the last place) leave about twenty. fp32 rows bring half as
// many values with their bytes and have room for the corrections that make
// both good to fp32's own precision.

#include "ep_experts.h"
#include "ep_gate.h"
#include "ep_quantise.h"

namespace epmi {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerCU = 64;
// Vectors of a block step, at least: a block takes as many whole rows at a
// time as hold them, so that narrow rows fill its lanes too.
constexpr int kStepVectors = 8 * kThreads;

// A thread takes 16 bytes of each half of a row. Rows are dealt in address
// order; row_src tells which hold a route, the others are zeroed under the
// layout's pad and tail policies. row_src is read one step ahead.
template <int DT, bool BWD>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(Dims d, HandleView hv, const row16_t* __restrict__ grad,
                  const row16_t* __restrict__ gate_up, row16_t* __restrict__ out,
                  int32_t step_rows) {
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  using P = Payload<DT>;
  constexpr int N = P::N;
  const int64_t live = hh.total < d.cap ? hh.total : d.cap;
  const int64_t rows = d.zero_tail ? d.cap : live;
  const int32_t V = (int32_t)d.V;
  // the thread's first place in a block step, and the way to its next one
  const int32_t row_first = threadIdx.x / V, v_first = threadIdx.x % V;
  const int32_t row_by = kThreads / V, v_by = kThreads % V;
  for (int64_t r0 = (int64_t)blockIdx.x * step_rows; r0 < rows;
       r0 += (int64_t)gridDim.x * step_rows) {
    const int64_t r1 = r0 + step_rows < rows ? r0 + step_rows : rows;
    int64_t r = r0 + row_first;
    int32_t v = v_first;
    int32_t source = r < r1 && r < live ? hv.row_src[r] : -1;
    while (r < r1) {
      int64_t next_r = r + row_by;
      int32_t next_v = v + v_by;
      if (next_v >= V) {
        next_v -= V;
        ++next_r;
      }
      const int32_t next_source = next_r < r1 && next_r < live ? hv.row_src[next_r] : -1;
      row16_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (source >= 0) {
        const row16_t gv = __builtin_nontemporal_load(gate_up + r * 2 * V + v);
        const row16_t uv = __builtin_nontemporal_load(gate_up + r * 2 * V + V + v);
        row16_t dv = {0, 0, 0, 0};
        if constexpr (BWD) dv = __builtin_nontemporal_load(grad + r * V + v);
        float o[N], o2[N];
        static_for<N>([&](auto j) {
          const float g = P::template get<j>(gv), u = P::template get<j>(uv);
          const Gate k = gate_of<DT == EP_DTYPE_FP32>(g);
          const float silu = g * k.p * k.r;   // but for one factor p
          if constexpr (BWD) {
            const float dd = P::template get<j>(dv);
            o[j] = dd * (k.p * (k.r * __builtin_fmaf(g, k.q, 1.f))) * (u * k.p);
            o2[j] = silu * (dd * k.p);
          } else {
            o[j] = silu * (u * k.p);
          }
        });
        a = pack<DT>(o);
        if constexpr (BWD) b = pack<DT>(o2);
      }
      if (source >= 0 || r >= live || d.fill_pads) {
        if constexpr (BWD) {
          store_stream16(out + r * 2 * V + v, a);
          store_stream16(out + r * 2 * V + V + v, b);
        } else {
          store_stream16(out + r * V + v, a);
        }
      }
      r = next_r;
      v = next_v;
      source = next_source;
    }
  }
}

// The activation with its result in 8 bits. The values of a scale lie side by
// side in a row: 16 (fp32: 32) neighbouring lanes hold them, 16 bytes of each
// half a lane, and the scale's maximum takes four (five) exchanges. Rows are
// dealt by such blocks in address order. 32768 rows of 14336 values 412 us, 5.8
// TB/s; uneven experts' 65536 rows of 768 47 to 53, by the calls around it; fp32,
// 16384 rows of 4096 110 us, 5.5 TB/s. Both of the first were bound by the arithmetic
// (420 and 51 us, beside 411 and 47 the same day) while a value took 32 vector
// instructions, for rows of a step in 64 bits, a shuffle an exchange, IEEE quotients
// and a flag a value: it takes 22.
template <int DT>
__global__ void __launch_bounds__(kThreads)
    swiglu_scaled_kernel(Dims d, HandleView hv, const row16_t* __restrict__ gate_up,
                         uint8_t* __restrict__ out_q, float* __restrict__ out_scales,
                         int32_t step_rows) {
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  using P = Payload<DT>;
  constexpr int N = P::N;
  constexpr int kLanes = kScaleBlock / N, kGroups = kThreads / kLanes;
  const int64_t live = hh.total < d.cap ? hh.total : d.cap;
  const int64_t rows = d.zero_tail ? d.cap : live;
  const int32_t V = (int32_t)d.V, S = (int32_t)EP_SCALE_COLUMNS(d.H);
  const int32_t B = (V + kLanes - 1) / kLanes;   // blocks of a row
  const int32_t group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int32_t row_first = group / B, b_first = group % B;
  const int32_t row_by = kGroups / B, b_by = kGroups % B;
  for (int64_t r0 = (int64_t)blockIdx.x * step_rows; r0 < rows;
       r0 += (int64_t)gridDim.x * step_rows) {
    // from here on rows and places count from r0 on: 32 bits hold a step's bytes
    auto of_step = [&](int64_t n) {
      return (int32_t)(n - r0 < 0 ? 0 : n - r0 < step_rows ? n - r0 : step_rows);
    };
    const int32_t here = of_step(rows), alive = of_step(live);
    const char* gate = reinterpret_cast<const char*>(gate_up + r0 * 2 * V);
    const char* up = gate + (int64_t)V * 16;
    uint8_t* to_q = out_q + r0 * d.H;
    char* to_scales = reinterpret_cast<char*>(out_scales + r0 * S);
    const char* sources = reinterpret_cast<const char*>(hv.row_src + r0);
    auto source_of = [&](int32_t r) {
      return r < alive ? *reinterpret_cast<const int32_t*>(sources + (uint32_t)r * 4) : -1;
    };
    int32_t r = row_first, b = b_first, source = source_of(r);
    while (r < here) {
      int32_t next_r = r + row_by, next_b = b + b_by;
      if (next_b >= B) {
        next_b -= B;
        ++next_r;
      }
      const int32_t next_source = source_of(next_r);
      const int32_t v = b * kLanes + lane;
      const bool in = v < V;
      uint32_t q[N / 4] = {};
      float scale = 0.f;
      if (source >= 0) {
        row16_t gv = {0, 0, 0, 0}, uv = {0, 0, 0, 0};
        if (in) {
          const uint32_t at = (uint32_t)(r * 2 * V + v) * 16;
          gv = __builtin_nontemporal_load(reinterpret_cast<const row16_t*>(gate + at));
          uv = __builtin_nontemporal_load(reinterpret_cast<const row16_t*>(up + at));
        }
        float o[N];
        static_for<N>([&](auto j) {
          const float g = P::template get<j>(gv);
          const Gate k = gate_of<DT == EP_DTYPE_FP32, true>(g);
          o[j] = g * k.p * k.r * (P::template get<j>(uv) * k.p);
        });
        scale = quantise<kLanes>(o, q);
      }
      if (source >= 0 || r >= alive || d.fill_pads) {
        if (in) store_bytes(to_q + (uint32_t)(r * V + v) * N, q);
        // with the last block, the columns past it too, fewer than eight
        if (lane == 0 || (b == B - 1 && lane < S - b))
          *reinterpret_cast<float*>(to_scales + (uint32_t)(r * S + b + lane) * 4) =
              lane == 0 ? scale : 0.f;
      }
      r = next_r;
      b = next_b;
      source = next_source;
    }
  }
}

}  // namespace

hipError_t launch_swiglu_scaled(const Dims& d, const HandleView& hv, const void* gate_up,
                                uint8_t* out_q, float* out_scales, int num_cus,
                                hipStream_t stream) {
  // Short blocks, of 512 vectors or a row, each of one step: 32768 rows of 14336 values
  // 410 us, 439 with two rows; uneven experts' rows of 768 53, and 61, 54 and 56 with
  // 256, 1024 and 2048 vectors. The limit keeps the grid's threads below 2^32.
  const int32_t step_rows = (int32_t)((512 + d.V - 1) / d.V);
  int64_t blocks = (d.cap + step_rows - 1) / step_rows;
  const int64_t most = (int64_t)num_cus * 4096;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  return with_payload(d.dtype, [&](auto dt) {
    swiglu_scaled_kernel<decltype(dt)::value><<<dim3((uint32_t)blocks), dim3(kThreads), 0, stream>>>(
        d, hv, static_cast<const row16_t*>(gate_up), out_q, out_scales, step_rows);
    return hipGetLastError();
  });
}

hipError_t launch_swiglu(const Dims& d, const HandleView& hv, bool backward, const void* grad,
                         const void* gate_up, void* out, int num_cus, hipStream_t stream) {
  const int32_t step_rows = (int32_t)((kStepVectors + d.V - 1) / d.V);
  int64_t blocks = (d.cap + step_rows - 1) / step_rows;
  const int64_t most = (int64_t)num_cus * kBlocksPerCU;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  return with_payload(d.dtype, [&](auto dt) {
    const dim3 grid((uint32_t)blocks), block(kThreads);
    const row16_t* g = static_cast<const row16_t*>(grad);
    const row16_t* gu = static_cast<const row16_t*>(gate_up);
    row16_t* o = static_cast<row16_t*>(out);
    if (backward) {
      swiglu_kernel<decltype(dt)::value, true>
          <<<grid, block, 0, stream>>>(d, hv, g, gu, o, step_rows);
    } else {
      swiglu_kernel<decltype(dt)::value, false>
          <<<grid, block, 0, stream>>>(d, hv, g, gu, o, step_rows);
    }
    return hipGetLastError();
  });
}

}  // namespace epmi
