// ep_layer.hip -- a whole expert layer for a few tokens, straight from the routing
// table: for every token t
//
//   result[t] = sum over its routes k, ascending, of
//               w[t, k] W_down[e] a(t, k),   a = silu(W_gate[e] x) * (W_up[e] x).
//
// Two kernels. A few tokens use each weight of the experts that they reach once,
// so these weights' bytes bound both; tiles of the two products stream them as
// ep_lines.h has it. What takes seven launches with a prepared routing needs
// neither its maps nor the expert-major rows: every block finds its expert and
// the expert's routes in the table itself, the rows of x are read where the tokens
// lie, and the activations and products are kept by route.

#include "ep_gate.h"
#include "ep_lines.h"

namespace epmi {

namespace {

constexpr int kMaxRoutes = EP_MAX_LAYER_ROUTES;
constexpr int kRowTile = 16;

// What a block works on: expert number `index` among those that have a route, in
// ascending order, and the routes of that expert, in ascending order too.
struct Routes {
  uint32_t has[kMaxExperts / 32];   // experts with a route
  uint16_t of[kMaxRoutes];          // expert of each route, kNone without one
  uint16_t rows[kMaxRoutes];        // the expert's routes
};
constexpr uint16_t kNone = 0xFFFF;
static_assert(kMaxExperts / 32 == kWave, "a word a lane");

struct Found {
  int32_t active;   // experts with a route
  int32_t expert;   // if index < active
  int32_t rows;
};

// Called by the whole block. Every wavefront writes all of r.rows, the same
// values, and so needs no barrier to read them.
template <int THREADS>
__device__ __forceinline__ Found find_expert(const int64_t* __restrict__ topk_idx, int32_t n,
                                             int32_t E, int32_t index, Routes& r) {
  const int lane = lane_id();
  if (threadIdx.x < kMaxExperts / 32) r.has[threadIdx.x] = 0;
  __syncthreads();
  for (int32_t s = threadIdx.x; s < n; s += THREADS) {
    const int64_t id = topk_idx[s];
    const bool valid = id >= 0 && id < E;
    r.of[s] = valid ? (uint16_t)id : kNone;
    if (valid) atomicOr(&r.has[id / 32], 1u << (id % 32));
  }
  __syncthreads();
  const uint32_t word = r.has[lane];
  const int32_t mine = __popc(word);
  int32_t sum = mine;
  static_for<6>([&](auto i) {
    const int32_t below = __shfl_up(sum, 1u << i, kWave);
    if (lane >= (1 << i)) sum += below;
  });
  Found f;
  f.active = __builtin_amdgcn_readlane(sum, kWave - 1);
  f.expert = 0;
  f.rows = 0;
  if (index >= f.active) return f;
  const uint64_t at = wave_ballot(sum - mine <= index && index < sum);
  const int word_lane = __builtin_ctzll(at);
  uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, word_lane);
  int32_t skip = index - __builtin_amdgcn_readlane(sum - mine, word_lane);
  while (skip-- > 0) bits &= bits - 1;
  f.expert = word_lane * 32 + __builtin_ctz(bits);
  for (int32_t s0 = 0; s0 < n; s0 += kWave) {
    const int32_t s = s0 + lane;
    const bool hit = s < n && r.of[s] == f.expert;
    const uint64_t hits = wave_ballot(hit);
    if (hit) r.rows[f.rows + __popcll(hits & ((1ull << lane) - 1))] = (uint16_t)s;
    f.rows += __popcll(hits);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return f;
}

// A tile's columns: COLS / 2 of gate and the same of up (UP), or COLS of the
// second product.
template <int F, int DT, int COLS, int WAVES, bool UP>
__global__ void __launch_bounds__(WAVES* kWave)
    layer_kernel(Dims d, LayerArgs a) {
  using S = Lines<F, DT, COLS>;
  constexpr int kThreads = WAVES * kWave, kHalf = COLS / 2;
  __shared__ __align__(16) char mem[WAVES * S::kLds];
  __shared__ Routes routes;
  __shared__ uint32_t last;
  const int32_t n = (int32_t)(d.T * d.K);
  const int32_t H = (int32_t)d.H, I = (int32_t)a.I;
  const int32_t K = UP ? H : I;                    // of this product
  const int32_t cols_all = UP ? I : H;             // columns of either half, or all
  if constexpr (UP) {
    // the second product's counters
    const int64_t all = (int64_t)gridDim.x * gridDim.y * kThreads;
    for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
         i < kLayerCounters; i += all)
      a.counters[i] = 0;
  }
  const int32_t n0 = blockIdx.x * (UP ? kHalf : COLS);
  const Found f = find_expert<kThreads>(a.topk_idx, n, d.E, blockIdx.y, routes);
  const int lane = lane_id(), i16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  char* lds = mem + wave * S::kLds;
  if (f.active == 0 && !UP && blockIdx.y == 0) {
    // no route at all: the result is zeros
    for (int32_t i = threadIdx.x; i < (int32_t)d.T * (COLS / 4); i += kThreads) {
      const int32_t t = i / (COLS / 4), c = n0 + i % (COLS / 4) * 4;
      if (c < H)
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.result) + (int64_t)t * H + c) =
            u32x2{0, 0};
    }
  }
  if ((int)blockIdx.y >= f.active) return;

  const int64_t e = f.expert;
  typename S::Source src;
  const char* w = static_cast<const char*>(UP ? a.gate_up : a.down);
  const int64_t w_row = (int64_t)K * S::kSize;
  const int64_t first = e * (UP ? 2 * (int64_t)I : H);   // first row of the expert's matrix
  src.w[0] = w + (first + n0) * w_row;
  if constexpr (UP) {
    src.cols[0] = src.cols[1] = I - n0 < kHalf ? I - n0 : kHalf;
    src.w[1] = src.w[0] + I * w_row;
  } else {
    const int32_t left = H - n0;
    src.cols[0] = left < kHalf ? left : kHalf;
    src.cols[1] = left < COLS ? left - src.cols[0] : kHalf;
    src.w[1] = src.w[0] + (src.cols[1] > 0 ? kHalf * w_row : 0);
  }
  if constexpr (F == kWeights8) {
    // the scales of the lane's four columns of each block of 16, which lie in one
    const int32_t KB = pieces(K, kScaleBlock);
    const int32_t NB = pieces(UP ? 2 * I : H, kScaleBlock);
    const float* scales = UP ? a.gate_up_scales : a.down_scales;
    static_for<S::kNF>([&](auto j) {
      constexpr int half = j / (S::kNF / 2);
      int32_t in = (j % (S::kNF / 2)) * 16 + q * 4;
      in = in < src.cols[half] ? in : 0;
      const int32_t c = n0 + (UP ? half * I : src.cols[half] > 0 ? half * kHalf : 0) + in;
      src.w_scales[j] = scales + (e * NB + c / kScaleBlock) * KB;
    });
  }
  S s;
  for (int32_t r0 = 0; r0 < f.rows; r0 += kRowTile) {
    const int32_t rows = f.rows - r0 < kRowTile ? f.rows - r0 : kRowTile;
    const int32_t route = routes.rows[r0 + (i16 < rows ? i16 : rows - 1)];
    src.x = UP ? static_cast<const char*>(a.tokens) + (int64_t)(route / d.K) * H * 2
               : static_cast<const char*>(a.act) + (int64_t)route * I * 2;
    s.first(src, wave, K);
    f32x4 acc[S::kNF];
    static_for<S::kNF>([&](auto j) { acc[j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    s.steps(lds, src, wave, WAVES, K, acc);
    S::put_sums(lds, acc);
    __syncthreads();
    // four columns of a row at a time
    constexpr int kQuads = (UP ? kHalf : COLS) / 4;
    for (int i = threadIdx.x; i < kRowTile * kQuads; i += kThreads) {
      const int m = i / kQuads, c = i % kQuads * 4;
      if (m < rows && n0 + c < cols_all) {
        const int64_t at = (int64_t)routes.rows[r0 + m] * cols_all + n0 + c;
        const f32x4 v = S::template sum_of<WAVES>(mem, m, c);
        if constexpr (UP) {
          const f32x4 u = S::template sum_of<WAVES>(mem, m, kHalf + c);
          f32x4 o;
          static_for<4>([&](auto k) {
            const Gate g = gate_of<false>(v[k.value]);
            o[k.value] = v[k.value] * g.p * g.r * (u[k.value] * g.p);
          });
          // the second product's operand: rounded to the payload type, as its
          // matrix instructions take it
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.act) + at) = round_four<DT>(o);
        } else {
          *reinterpret_cast<f32x4*>(a.y + at) = v;
        }
      }
    }
    __syncthreads();
  }
  if constexpr (!UP) {
    // The last block of these columns adds up every token's routes, in ascending
    // order whichever block that is.
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
      last = atomicAdd(&a.counters[blockIdx.x], 1u) == (uint32_t)f.active - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int32_t i = threadIdx.x; i < (int32_t)d.T * (COLS / 4); i += kThreads) {
      const int32_t t = i / (COLS / 4), c = n0 + i % (COLS / 4) * 4;
      if (c >= H) continue;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      bool any = false;
      for (int32_t k = 0; k < d.K; ++k) {
        const int32_t route = t * d.K + k;
        if (routes.of[route] == kNone) continue;
        const f32x4 y = *reinterpret_cast<const f32x4*>(a.y + (int64_t)route * H + c);
        const float wk = a.topk_weights[route];
        static_for<4>([&](auto j) {
          sum[j.value] = any ? __builtin_fmaf(wk, y[j.value], sum[j.value]) : wk * y[j.value];
        });
        any = true;
      }
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.result) + (int64_t)t * H + c) =
          round_four<DT>(sum);
    }
  }
}

template <int F, int DT>
hipError_t launch_layer(const Dims& d, const LayerArgs& a, hipStream_t stream) {
  constexpr int kCols = 64, kWaves = 4;
  const int64_t n = d.T * d.K;
  const uint32_t experts = (uint32_t)(n < d.E ? n : d.E);
  layer_kernel<F, DT, kCols, kWaves, true>
      <<<dim3((uint32_t)((a.I + kCols / 2 - 1) / (kCols / 2)), experts), dim3(kWaves * kWave), 0,
         stream>>>(d, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  layer_kernel<F, DT, kCols, kWaves, false>
      <<<dim3((uint32_t)((d.H + kCols - 1) / kCols), experts), dim3(kWaves * kWave), 0, stream>>>(
          d, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_layer(const Dims& d, const LayerArgs& a, int, hipStream_t stream) {
  const bool eight = a.gate_up_scales != nullptr;
  if (d.dtype == EP_DTYPE_FP16)
    return eight ? launch_layer<kWeights8, EP_DTYPE_FP16>(d, a, stream)
                 : launch_layer<kPayload, EP_DTYPE_FP16>(d, a, stream);
  return eight ? launch_layer<kWeights8, EP_DTYPE_BF16>(d, a, stream)
               : launch_layer<kPayload, EP_DTYPE_BF16>(d, a, stream);
}

}  // namespace epmi
