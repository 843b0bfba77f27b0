// ep_scaled.h -- values in 8 bits: e4m3 with one fp32 scale for every 128 values
// of a row (weights: for every 128 x 128), and the launchers of the kernels that
// make and use them and of the ones around them (norm, layer for a few tokens).
//
//   scale = max(amax, 448 * 2^-100) / 448,  q = e4m3(y * (1 / scale))
//
// amax is that of a block's finite values: an infinity or NaN becomes a NaN of
// its own place and leaves its neighbours as they are. 448 is e4m3's largest
// value, so no finite value is cut off; the floor keeps a scale a normal number
// whose reciprocal is finite, also of a block of zeros or subnormals.
#pragma once

#include "ep.h"
#include "ep_internal.h"

namespace epmi {

constexpr int kScaleBlock = EP_SCALE_BLOCK;
constexpr float kE4m3Max = 448.f;
constexpr float kLeastAmax = 448.f * 0x1p-100f;

// The norm in front of a layer and its gradient (ep_norm.hip), T rows of H.
struct NormArgs {
  const void* x;
  const void* residual;     // or null
  const void* weight;
  void* sum;                // x + residual, with a residual
  void* out;                // payload rows, or null
  uint8_t* out_q;           // e4m3 rows with their scales, or null
  float* out_scales;
  float eps;
};
hipError_t launch_rms_norm(const Dims& d, const NormArgs& a, hipStream_t stream);

struct NormBwdArgs {
  const void* grad;
  const void* grad_sum;     // or null
  const void* x;
  const void* weight;
  void* grad_x;
  void* grad_weight;        // or null
  float* partial;           // norm_bwd_partials(T, H, dtype) rows of H
  float eps;
};
// Rows of partial weight gradients: one for each block, a number that the layout
// alone fixes.
int64_t norm_bwd_partials(const Dims& d);
hipError_t launch_rms_norm_bwd(const Dims& d, const NormBwdArgs& a, hipStream_t stream);

// The gated activation with its result in 8 bits (ep_swiglu.hip).
hipError_t launch_swiglu_scaled(const Dims& d, const HandleView& hv, const void* gate_up,
                                uint8_t* out_q, float* out_scales, int num_cus,
                                hipStream_t stream);

// The grouped product of 8-bit operands (ep_scaled.hip).
hipError_t launch_grouped_scaled(const Dims& d, const HandleView& hv, const uint8_t* x,
                                 const float* x_scales, const uint8_t* w, const float* w_scales,
                                 void* out, int64_t N, int num_cus, hipStream_t stream);

// The whole layer for a few tokens (ep_layer.hip).
struct LayerArgs {
  const int64_t* topk_idx;
  const float* topk_weights;
  const void* tokens;
  const void* gate_up;          // [E, 2I, H], payload or e4m3
  const float* gate_up_scales;  // null for payload weights
  const void* down;             // [E, H, I]
  const float* down_scales;
  void* result;
  // the workspace's parts: one counter for each column tile of the second
  // product, activations [2, T*K, I] as sums of two values of the payload type, in
  // fp16 times a power of two for every 16 (exponent bytes [T*K, ceil(I/128) * 8]),
  // products [T*K, H]
  uint32_t* counters;
  void* act;
  uint8_t* act_exps;
  float* y;
  int64_t I;
};
constexpr int kLayerCounters = EP_MAX_FEATURES / 32;
hipError_t launch_expert_layer(const Dims& d, const LayerArgs& a, int num_cus,
                               hipStream_t stream);

}  // namespace epmi
