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
// lie, and the activations and products are kept by route. One token by top-2 of 8,
// 4096 x 14336, bf16: 115 us, 6.1 TB/s; 16 tokens by top-8 of 256, 7168 x 2048, 8
// bits: 682 to 720, 6.2 to 6.6 TB/s.

#include "ep_gate.h"
#include "ep_lines.h"

namespace epmi {

namespace {

constexpr int kMaxRoutes = EP_MAX_LAYER_ROUTES;
// Rows of x that a matrix instruction takes, and routes of an expert that a tile
// has: as many in the first product, half in the second, where a route's
// activations are two rows (see below).
constexpr int kRows = 16;
template <bool UP>
constexpr int kRoutes = UP ? kRows : kRows / 2;

// The routing table in LDS: the expert of each route, kNone without a valid one,
// and a bit for each expert that has a route.
struct Routes {
  uint32_t has[kMaxExperts / 32];
  uint16_t of[kMaxRoutes];
};
constexpr uint16_t kNone = 0xFFFF;
static_assert(kMaxExperts / 32 == kWave, "a word a lane");

// What a wavefront keeps of it: the experts with a route, in ascending order.
struct Active {
  uint32_t word;     // this lane's 32 experts
  int32_t before;    // experts with a route in the lanes below
  int32_t all;

  // Called by the whole block.
  template <int THREADS>
  __device__ static __forceinline__ Active of(const int64_t* __restrict__ topk_idx, int32_t n,
                                              int32_t E, Routes& r) {
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
    Active a;
    a.word = r.has[lane];
    int32_t sum = __popc(a.word);
    static_for<6>([&](auto i) {
      const int32_t below = __shfl_up(sum, 1u << i, kWave);
      if (lane >= (1 << i)) sum += below;
    });
    a.all = __builtin_amdgcn_readlane(sum, kWave - 1);
    a.before = sum - __popc(a.word);
    return a;
  }

  // Expert number `index` of them.
  __device__ __forceinline__ int32_t expert(int32_t index) const {
    const uint64_t at = wave_ballot(before <= index && index < before + __popc(word));
    const int from = __builtin_ctzll(at);
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, from);
    int32_t skip = index - __builtin_amdgcn_readlane(before, from);
    while (skip-- > 0) bits &= bits - 1;
    return from * 32 + __builtin_ctz(bits);
  }
};

// The expert's routes in ascending order: how many, and number first + i of them
// in each lane i below ROUTES (and so in i + ROUTES and on), as far as there are;
// the last one beyond. `mine` is the wavefront's own.
template <int ROUTES>
__device__ __forceinline__ int32_t routes_of(const Routes& r, int32_t n, int32_t expert,
                                             int32_t first, uint16_t (&mine)[kRows],
                                             int32_t& route) {
  const int lane = lane_id();
  int32_t rows = 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int32_t s0 = 0; s0 < n; s0 += kWave) {
    const int32_t s = s0 + lane;
    const bool hit = s < n && r.of[s] == expert;
    const uint64_t hits = wave_ballot(hit);
    const int32_t at = rows + __popcll(hits & ((1ull << lane) - 1)) - first;
    if (hit && at >= 0 && at < ROUTES) mine[at] = (uint16_t)s;
    rows += __popcll(hits);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int32_t last = rows - first < ROUTES ? rows - first - 1 : ROUTES - 1;
  const int32_t i = lane % ROUTES;
  route = mine[i < last ? i : last];
  return rows;
}

// Four products of a route, written by one block and read by another, perhaps on
// another XCD with an L2 of its own: stores and loads of agent scope, which go
// through to the memory that the XCDs share. The fences that plain accesses would
// need write back and invalidate a whole L2 for every block: with an
// acquire-release add the second product took 802 us in place of 257 (batch of 16,
// 256 experts of 7168 x 2048), with a fence in every thread 2442.
__device__ __forceinline__ void put_product(float* to, f32x4 v) {
  uint64_t* p = reinterpret_cast<uint64_t*>(to);
  static_for<2>([&](auto i) {
    const uint64_t bits = (uint64_t)__float_as_uint(v[2 * i.value]) |
                          (uint64_t)__float_as_uint(v[2 * i.value + 1]) << 32;
    __hip_atomic_store(p + i, bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  });
}
__device__ __forceinline__ f32x4 get_product(const float* from) {
  const uint64_t* p = reinterpret_cast<const uint64_t*>(from);
  f32x4 v;
  static_for<2>([&](auto i) {
    const uint64_t bits = __hip_atomic_load(p + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v[2 * i.value] = __uint_as_float((uint32_t)bits);
    v[2 * i.value + 1] = __uint_as_float((uint32_t)(bits >> 32));
  });
  return v;
}

// A tile is up to kRoutes routes of an expert by COLS / 2 columns of gate and the same of
// up (UP), or by COLS columns of the second product. The wavefronts take the steps
// of k in turn and add their sums in LDS at the end, by when each has the first
// loads of the block's next tile in flight. An expert's row tiles follow each
// other in one block.
template <int F, int DT, int COLS, int WAVES, bool UP>
__global__ void __launch_bounds__(WAVES* kWave)
    layer_kernel(Dims d, LayerArgs a) {
  constexpr bool kExps = DT == EP_DTYPE_FP16;      // of the activations
  using S = Lines<F, DT, COLS, !UP && kExps>;
  constexpr int kThreads = WAVES * kWave, kHalf = COLS / 2;
  constexpr int kTileCols = UP ? kHalf : COLS, kQuads = kTileCols / 4;
  constexpr int kTile = kRoutes<UP>;
  extern __shared__ __align__(16) char mem[];      // WAVES * S::kLds
  __shared__ Routes routes;
  __shared__ uint16_t row_lists[WAVES][kRows];
  __shared__ uint32_t last;
  const int32_t n = (int32_t)(d.T * d.K);
  const int32_t H = (int32_t)d.H, I = (int32_t)a.I;
  const int32_t K = UP ? H : I;                    // of this product
  const int32_t cols_all = UP ? I : H;             // columns of either half, or all
  const int64_t exps_row = pieces(I, kScaleBlock) * (kScaleBlock / kExpGroup);
  if constexpr (UP) {
    // the second product's counters, one for each of its column tiles at most
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces(H, 32);
         i += (int64_t)gridDim.x * kThreads)
      a.counters[i] = 0;
  }
  const Active active = Active::of<kThreads>(a.topk_idx, n, d.E, routes);
  const int lane = lane_id(), i16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  char* lds = mem + wave * S::kLds;
  const int32_t ct = (cols_all + kTileCols - 1) / kTileCols;
  const int32_t tiles = active.all * ct;

  // Every token's routes added up, ascending, in the columns from n0 on.
  auto add_up = [&](int32_t n0) {
    for (int32_t i = threadIdx.x; i < (int32_t)d.T * kQuads; i += kThreads) {
      const int32_t t = i / kQuads, c = n0 + i % kQuads * 4;
      if (c >= H) continue;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      bool any = false;
      for (int32_t k = 0; k < d.K; ++k) {
        const int32_t route = t * d.K + k;
        if (routes.of[route] == kNone) continue;
        const f32x4 y = get_product(a.y + (int64_t)route * H + c);
        const float wk = a.topk_weights[route];
        static_for<4>([&](auto j) {
          sum[j.value] = any ? __builtin_fmaf(wk, y[j.value], sum[j.value]) : wk * y[j.value];
        });
        any = true;
      }
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.result) + (int64_t)t * H + c) =
          round4<DT>(sum);
    }
  };
  if constexpr (!UP) {
    // no route at all: zeros
    if (tiles == 0)
      for (int32_t t = blockIdx.x; t < ct; t += gridDim.x) add_up(t * COLS);
  }

  struct Place {
    typename S::Source src;
    int32_t tile, n0;
    int32_t first, rows;   // first of the tile's routes, routes of the expert
    int32_t route;         // of the lane's row
  };
  // Starts the loads of a tile: the weights', whose place the expert tells, before
  // the expert's routes are looked up.
  S s;
  auto start = [&](int32_t tile, int32_t first) {
    Place p;
    p.tile = tile;
    p.first = first;
    const int32_t e = active.expert(tile / ct);
    p.n0 = tile % ct * kTileCols;
    const char* w = static_cast<const char*>(UP ? a.gate_up : a.down);
    const int64_t w_row = (int64_t)K * S::kSize;
    const int64_t row = (int64_t)e * (UP ? 2 * (int64_t)I : H) + p.n0;
    const int32_t left = cols_all - p.n0;
    p.src.w[0] = w + row * w_row;
    p.src.cols[0] = left < kHalf ? left : kHalf;
    if constexpr (UP) {
      p.src.cols[1] = p.src.cols[0];
      p.src.w[1] = p.src.w[0] + I * w_row;
    } else {
      p.src.cols[1] = left < COLS ? left - p.src.cols[0] : kHalf;
      p.src.w[1] = p.src.w[0] + (p.src.cols[1] > 0 ? kHalf * w_row : 0);
    }
    if constexpr (F == kWeights8) {
      // the scales of the lane's four columns of each block of 16, which lie in one
      const int32_t KB = pieces(K, kScaleBlock);
      const int32_t NB = pieces(UP ? 2 * I : H, kScaleBlock);
      const float* scales = (UP ? a.gate_up_scales : a.down_scales) + (int64_t)e * NB * KB;
      static_for<S::kNF>([&](auto j) {
        constexpr int half = j / (S::kNF / 2);
        int32_t in = (j % (S::kNF / 2)) * 16 + q * 4;
        in = in < p.src.cols[half] ? in : 0;
        const int32_t c = p.n0 + (UP ? half * I : p.src.cols[half] > 0 ? half * kHalf : 0) + in;
        p.src.w_scales[j] = scales + (int64_t)(c / kScaleBlock) * KB;
      });
    }
    const bool mine = wave < K / S::kStep;
    if (mine) s.template load_weights<false>(p.src, wave * S::kStep, K);
    p.rows = routes_of<kTile>(routes, n, e, first, row_lists[wave], p.route);
    // the second product: the high parts of eight routes' activations in the rows,
    // then the low ones
    p.src.x = UP ? static_cast<const char*>(a.tokens) + (int64_t)(p.route / d.K) * H * 2
                 : static_cast<const char*>(a.act) +
                       (int64_t)(p.route + (i16 < kTile ? 0 : n)) * I * 2;
    if constexpr (!UP && kExps) p.src.x_exps = a.act_exps + p.route * exps_row;
    if (mine) s.template load_x<false>(p.src, wave * S::kStep, K);
    return p;
  };
  // UP = false: the tile whose products are on their way, its columns' counter not
  // yet raised
  int32_t pending = -1;
  auto raise = [&]() {
    if (threadIdx.x == 0)
      last = pending >= 0 &&
             __hip_atomic_fetch_add(&a.counters[pending], 1u, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)active.all - 1;
  };

  Place next;
  next.tile = blockIdx.x;
  if (next.tile < tiles) next = start(next.tile, 0);
  while (next.tile < tiles) {
    const Place cur = next;
    f32x4 acc[S::kNF];
    static_for<S::kNF>([&](auto j) { acc[j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    s.steps(lds, cur.src, wave, WAVES, K, acc);
    // the last tile's products have been acknowledged (all loads are used up: this
    // waits for nothing else)
    if constexpr (!UP) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const bool done = cur.first + kTile >= cur.rows;   // of this tile's expert
    const int32_t rows = done ? cur.rows - cur.first : kTile;
    next.tile = done ? cur.tile + (int32_t)gridDim.x : cur.tile;
    if (next.tile < tiles) next = start(next.tile, done ? 0 : cur.first + kTile);
    S::put_sums(lds, acc);
    __syncthreads();
    if constexpr (!UP) raise();
    // four columns of a row at a time
    for (int i = threadIdx.x; i < kTile * kQuads; i += kThreads) {
      const int m = i / kQuads, c = i % kQuads * 4;
      const int32_t route = __shfl(cur.route, m, kWave);
      const bool there = m < rows && cur.n0 + c < cols_all;
      const int64_t at = (int64_t)route * cols_all + cur.n0 + c;
      if constexpr (UP) {
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        if (there) {
          const f32x4 v = S::template sum_of<WAVES>(mem, m, c);
          const f32x4 u = S::template sum_of<WAVES>(mem, m, kHalf + c);
          static_for<4>([&](auto k) {
            const Gate g = gate_of<false>(v[k.value]);
            o[k.value] = v[k.value] * g.p * g.r * (u[k.value] * g.p);
          });
        }
        // The second product's operand: its matrix instructions take the payload
        // type, so an activation is kept as the sum of two such values, each a row
        // of it. Rounded to one, it would add as much to the result's error as that's
        // own rounding. An expert has few routes: the rows are there anyway. Two bf16
        // values hold 16 bits of any fp32 number; two of fp16 hold 22 bits in a part
        // of its range, to which each 16 of a route are brought by a power of two.
        if constexpr (kExps) {
          static_assert(!UP || kTileCols == kExpGroup, "a tile's columns share an exponent");
          float amax = 0.f;    // past a NaN; an infinity stays one
          static_for<4>([&](auto k) {
            amax = __builtin_fmaxf(amax, __builtin_fabsf(o[k.value]));
          });
          static_for<2>([&](auto i) {
            amax = __builtin_fmaxf(amax, __shfl_xor(amax, 1 << i, kWave));
          });
          const uint32_t e = exponent_for(amax);
          o *= inverse_power_of(e);
          if (there && c == 0)
            a.act_exps[route * exps_row + cur.n0 / kExpGroup] = (uint8_t)e;
        }
        if (there) {
          const u32x2 high = round4<DT>(o);
          f32x4 rest;
          static_for<4>([&](auto k) {
            const uint32_t bits = (high[k.value / 2] >> (k.value % 2 * 16)) & 0xFFFFu;
            const float h = DT == EP_DTYPE_BF16 ? __uint_as_float(bits << 16) : f16_to_f32(bits);
            // past the type's range, and NaN: nothing to add
            rest[k.value] = __builtin_fabsf(h) < __builtin_inff() ? o[k.value] - h : 0.f;
          });
          uint16_t* act = static_cast<uint16_t*>(a.act) + at;
          *reinterpret_cast<u32x2*>(act) = high;
          *reinterpret_cast<u32x2*>(act + (int64_t)n * I) = round4<DT>(rest);
        }
      } else if (there) {
        put_product(a.y + at, S::template sum_of<WAVES>(mem, m, c) +
                                  S::template sum_of<WAVES>(mem, kTile + m, c));
      }
    }
    __syncthreads();
    if constexpr (!UP) {
      if (last) add_up(pending * COLS);
      pending = done ? cur.tile % ct : -1;
    }
  }
  if constexpr (!UP) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    raise();
    __syncthreads();
    if (last) add_up(pending * COLS);
  }
}

template <int F, int DT, bool UP, int COLS, int WAVES>
hipError_t launch_product(const Dims& d, const LayerArgs& a, int64_t blocks, hipStream_t stream) {
  constexpr int kTileCols = UP ? COLS / 2 : COLS;
  const int64_t routes = d.T * d.K, cols = UP ? a.I : d.H;
  // the most experts that the routes can reach
  const int64_t tiles = (routes < d.E ? routes : d.E) * ((cols + kTileCols - 1) / kTileCols);
  if (blocks > tiles) blocks = tiles;
  layer_kernel<F, DT, COLS, WAVES, UP>
      <<<dim3((uint32_t)blocks), dim3(WAVES * kWave), WAVES * Lines<F, DT, COLS>::kLds, stream>>>(
          d, a);
  return hipGetLastError();
}

// Columns of a tile and wavefronts that share its k; times of the two products
// together, from one captured graph, weights out of HBM.
//   16 bits, both products: 32 columns and eight wavefronts, two blocks a CU. Against
//   64 columns and four wavefronts, four blocks: one token by top-2 of 8, 4096 x
//   14336, 135 against 146 us (first product) and 126 against 146 (second); 16
//   tokens by top-8 of 128, 2048 x 768, 139 and 145 against 149; 8 tokens of the
//   first layer 380 and 407 against 405.
//   8 bits, first product: 32 columns and four wavefronts, eight blocks: one token of
//   the first layer 86 against 91, 16 tokens by top-8 of 256, 7168 x 2048, 699
//   against 705 (64 tokens 1556 against 1544).
//   8 bits, second product: 64 columns and four wavefronts, four blocks (with 32 and
//   eight the 16 tokens take 782 against 703, their 16 steps of k being two a
//   wavefront), but 32 and eight where tiles of 64 leave CUs without work: one token
//   of the first layer 68 against 86.
template <int F, int DT>
hipError_t launch_layer(const Dims& d, const LayerArgs& a, int num_cus, hipStream_t stream) {
  const int64_t cus = num_cus, routes = d.T * d.K;
  if constexpr (F == kPayload) {
    const hipError_t e = launch_product<F, DT, true, 32, 8>(d, a, 2 * cus, stream);
    return e != hipSuccess ? e : launch_product<F, DT, false, 32, 8>(d, a, 2 * cus, stream);
  } else {
    const hipError_t e = launch_product<F, DT, true, 32, 4>(d, a, 8 * cus, stream);
    if (e != hipSuccess) return e;
    if ((routes < d.E ? routes : d.E) * ((d.H + 63) / 64) < cus)
      return launch_product<F, DT, false, 32, 8>(d, a, 2 * cus, stream);
    return launch_product<F, DT, false, 64, 4>(d, a, 4 * cus, stream);
  }
}

}  // namespace

hipError_t launch_expert_layer(const Dims& d, const LayerArgs& a, int num_cus,
                               hipStream_t stream) {
  const bool eight = a.gate_up_scales != nullptr;
  if (d.dtype == EP_DTYPE_FP16)
    return eight ? launch_layer<kWeights8, EP_DTYPE_FP16>(d, a, num_cus, stream)
                 : launch_layer<kPayload, EP_DTYPE_FP16>(d, a, num_cus, stream);
  return eight ? launch_layer<kWeights8, EP_DTYPE_BF16>(d, a, num_cus, stream)
               : launch_layer<kPayload, EP_DTYPE_BF16>(d, a, num_cus, stream);
}

}  // namespace epmi
