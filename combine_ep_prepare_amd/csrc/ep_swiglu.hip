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

namespace epmi {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerCU = 64;
// Vectors of a block step, at least: a block takes as many whole rows at a
// time as hold them, so that narrow rows fill its lanes too.
constexpr int kStepVectors = 8 * kThreads;

// What the results take from a gate g. With e = exp(-|g|) and r = 1 / (1 + e),
//   s = 1 / (1 + exp(-g)) = p^2 r and 1 - s = q, where
//   p = 1, q = e r for g >= 0 and p = sqrt(e), q = r for g < 0:
// no exponential overflows, 1 - s does not cancel, and s enters a product as
// one p a factor, so that a sigmoid below fp32's range still counts: a gate of
// -88 gives silu(g) = -5e-37. p is a normal number down to g = -174, past which
// it is 0.
struct Gate {
  float p, q, r;
};

// The exponent |g| log2(e) / 2 of p is rounded, which takes p off by up to
// |g| / 2 units of 2^-24: nothing to a 16-bit result (a gate of 174 makes 2^-16
// of it in s). EXACT, for fp32, carries what the rounding and the constant
// leave out into p and refines the reciprocal by a step: s is then within 20
// units of 2^-24 of its value at any g, in the time that the rows' bytes take
// anyway (8192 rows by top-2, 4096 values out: 146 us with it and without).
template <bool EXACT>
__device__ __forceinline__ Gate gate_of(float g) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHi = (float)kLog2e, kLo = (float)(kLog2e - (double)kHi);
  constexpr float kHalfLn2 = 0.34657359027997265f;
  Gate o;
  float root;   // sqrt(e)
  if constexpr (EXACT) {
    // past 400 p is 0, and an infinite g would make the rest a NaN
    const float x = __builtin_fminf(__builtin_fabsf(g), 400.f);
    const float a = x * kHi;
    const float rest = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -a));
    root = __builtin_amdgcn_exp2f(a * -0.5f);
    root = __builtin_fmaf(root, rest * -kHalfLn2, root);
  } else {
    root = __builtin_amdgcn_exp2f(__builtin_fabsf(g) * (-0.5f * kHi));
  }
  const float e = root * root, d = 1.f + e;
  o.r = __builtin_amdgcn_rcpf(d);
  if constexpr (EXACT) o.r = __builtin_fmaf(__builtin_fmaf(-d, o.r, 1.f), o.r, o.r);
  o.p = g < 0.f ? root : 1.f;
  o.q = g < 0.f ? o.r : e * o.r;
  return o;
}

// Rounds like Payload::pack; where no lane has a NaN, by the hardware's packed
// conversions.
template <int DT, int N>
__device__ __forceinline__ row16_t pack(const float (&o)[N]) {
  if constexpr (DT != EP_DTYPE_FP32) {
    bool nan = false;
    static_for<N / 2>([&](auto j) { nan |= __builtin_isunordered(o[2 * j], o[2 * j + 1]); });
    if (wave_ballot(nan) == 0) {
      typedef std::conditional_t<DT == EP_DTYPE_BF16, __bf16, _Float16> half;
      typedef half half2 __attribute__((ext_vector_type(2)));
      typedef float float2v __attribute__((ext_vector_type(2)));
      row16_t v;
      static_for<4>([&](auto j) {
        float2v f = {o[2 * j], o[2 * j + 1]};
        // the fp32 results stand as they are: no fusing of the last product
        // with the conversion, which would skip its rounding
        asm("" : "+v"(f));
        v[j.value] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, half2));
      });
      return v;
    }
  }
  return Payload<DT>::pack(o);
}

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

}  // namespace

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
