// ep_norm.hip -- the root-mean-square norm in front of an expert layer, with the
// residual's addition, a result in the payload type or in 8 bits with scales, and
// its gradient.
//
//   s = x + residual (rounded to the payload type: it is an output, and the norm
//       is that of the rounded values, so that the backward pass, which reads
//       them, differentiates what was computed)
//   y = s * r * w,  r = 1 / sqrt(mean(s^2) + eps)
//
//   with n = s r and c = mean(grad * w * n):
//   grad_s = r (grad * w - n c) (+ grad_sum),  grad_w = sum over rows of grad * n
//
// Both are bound by HBM traffic. A row is read once and stays in registers
// between its sums and its results: a wavefront holds rows of up to 256 16-byte
// vectors, a block of four to sixteen wavefronts longer ones. Sums are fp32. 32768
// rows of 7168 bf16 values with a residual, in 8 bits: 268 us, 6.2 TB/s; the gradient
// of 16384 rows of 4096 with one of the sum: 92 us, 5.9 TB/s, 5 of them the sum of
// the blocks' parts.

#include "ep_experts.h"
#include "ep_gate.h"
#include "ep_matrix.h"
#include "ep_quantise.h"

namespace epmi {

namespace {

// Adds N sums over the block's WAVES wavefronts (over the wavefront for one).
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&sums)[N], float* lds) {
  static_for<6>([&](auto i) {
    static_for<N>([&](auto n) { sums[n] += __shfl_xor(sums[n], 1 << i, kWave); });
  });
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x / kWave;
    if (lane_id() == 0) static_for<N>([&](auto n) { lds[n * WAVES + wave] = sums[n]; });
    __syncthreads();
    static_for<N>([&](auto n) { sums[n] = 0.f; });
    static_for<WAVES>([&](auto w) {
      static_for<N>([&](auto n) { sums[n] += lds[n * WAVES + w]; });
    });
  }
}

__device__ __forceinline__ float inverse_rms(float sum, int64_t H, float eps) {
  return 1.f / __builtin_sqrtf(sum / (float)H + eps);
}

// Rows of a block (of 256 threads at least): one a wavefront, or one.
constexpr int rows_of_block(int waves) { return waves == 1 ? 4 : 1; }
constexpr int threads_of_block(int waves) { return (waves == 1 ? 4 : waves) * kWave; }

template <int DT, int WAVES, int VPT>
__global__ void __launch_bounds__(threads_of_block(WAVES))
    rms_norm_kernel(Dims d, NormArgs a) {
  using P = Payload<DT>;
  constexpr int N = P::N;
  constexpr int kLanes = kScaleBlock / N;   // lanes that hold a block of values
  __shared__ float lds[WAVES];
  const int t = WAVES == 1 ? lane_id() : (int)threadIdx.x;
  const int64_t row = WAVES == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / kWave
                                 : (int64_t)blockIdx.x;
  if (row >= d.T) return;   // with one wavefront a row: no barrier follows
  const int32_t V = (int32_t)d.V;
  const row16_t* x = static_cast<const row16_t*>(a.x) + row * V;
  const row16_t* res = static_cast<const row16_t*>(a.residual) + row * V;
  const row16_t* weight = static_cast<const row16_t*>(a.weight);
  row16_t s[VPT], w[VPT];
  static_for<VPT>([&](auto i) {
    const int v = i * (WAVES * kWave) + t;
    s[i] = row16_t{0, 0, 0, 0};
    if (v < V) s[i] = __builtin_nontemporal_load(x + v);
  });
  // asked for with the rows: the stores below keep later loads behind them
  static_for<VPT>([&](auto i) {
    const int v = i * (WAVES * kWave) + t;
    w[i] = row16_t{0, 0, 0, 0};
    if (v < V) w[i] = weight[v];
  });
  if (a.residual) {
    row16_t b[VPT];
    static_for<VPT>([&](auto i) {
      const int v = i * (WAVES * kWave) + t;
      b[i] = row16_t{0, 0, 0, 0};
      if (v < V) b[i] = __builtin_nontemporal_load(res + v);
    });
    static_for<VPT>([&](auto i) {
      float o[N];
      static_for<N>([&](auto j) {
        o[j] = P::template get<j>(s[i]) + P::template get<j>(b[i]);
      });
      s[i] = pack<DT>(o);
      const int v = i * (WAVES * kWave) + t;
      if (v < V) store_stream16(static_cast<row16_t*>(a.sum) + row * V + v, s[i]);
    });
  }
  float ss[1] = {0.f};
  static_for<VPT>([&](auto i) {
    static_for<N>([&](auto j) {
      const float f = P::template get<j>(s[i]);
      ss[0] = __builtin_fmaf(f, f, ss[0]);
    });
  });
  row_sums<WAVES>(ss, lds);
  const float r = inverse_rms(ss[0], d.H, a.eps);
  static_for<VPT>([&](auto i) {
    const int v = i * (WAVES * kWave) + t;
    float y[N];
    static_for<N>([&](auto j) {
      y[j] = P::template get<j>(s[i]) * r * P::template get<j>(w[i]);
    });
    if (a.out) {
      const row16_t o = pack<DT>(y);
      if (v < V) store_stream16(static_cast<row16_t*>(a.out) + row * V + v, o);
    }
    if (a.out_q) {
      // lanes past the row hold zeros
      uint32_t q[N / 4];
      const float scale = quantise<kLanes>(y, q);
      const int64_t S = EP_SCALE_COLUMNS(d.H);
      if (v < V) {
        store_bytes(a.out_q + row * d.H + (int64_t)v * N, q);
        if (v % kLanes == 0) a.out_scales[row * S + v / kLanes] = scale;
      }
    }
  });
  if (a.out_q) {
    // the columns past the row's blocks, fewer than eight
    const int64_t S = EP_SCALE_COLUMNS(d.H), blocks = (d.H + kScaleBlock - 1) / kScaleBlock;
    if (t < S - blocks) a.out_scales[row * S + blocks + t] = 0.f;
  }
}

template <int DT, int WAVES, int VPT>
__global__ void __launch_bounds__(threads_of_block(WAVES))
    rms_norm_bwd_kernel(Dims d, NormBwdArgs a) {
  using P = Payload<DT>;
  constexpr int N = P::N, kRows = rows_of_block(WAVES);
  __shared__ float lds[2 * 2 * WAVES];
  const int t = WAVES == 1 ? lane_id() : (int)threadIdx.x;
  const int64_t slot = (int64_t)blockIdx.x * kRows + (WAVES == 1 ? threadIdx.x / kWave : 0);
  const int32_t V = (int32_t)d.V;
  row16_t w[VPT];
  float dw[VPT][N];
  static_for<VPT>([&](auto i) {
    const int v = i * (WAVES * kWave) + t;
    w[i] = row16_t{0, 0, 0, 0};
    if (v < V) w[i] = static_cast<const row16_t*>(a.weight)[v];
    static_for<N>([&](auto j) { dw[i][j] = 0.f; });
  });
  int turn = 0;
  for (int64_t row = slot; row < d.T; row += (int64_t)gridDim.x * kRows) {
    const row16_t* x = static_cast<const row16_t*>(a.x) + row * V;
    const row16_t* grad = static_cast<const row16_t*>(a.grad) + row * V;
    const row16_t* more = static_cast<const row16_t*>(a.grad_sum) + row * V;
    row16_t s[VPT], g[VPT], m[VPT];
    static_for<VPT>([&](auto i) {
      const int v = i * (WAVES * kWave) + t;
      s[i] = g[i] = m[i] = row16_t{0, 0, 0, 0};
      if (v < V) {
        s[i] = __builtin_nontemporal_load(x + v);
        g[i] = __builtin_nontemporal_load(grad + v);
        if (a.grad_sum) m[i] = __builtin_nontemporal_load(more + v);
      }
    });
    float sums[2] = {0.f, 0.f};   // of s^2, and of grad * w * s
    static_for<VPT>([&](auto i) {
      static_for<N>([&](auto j) {
        const float f = P::template get<j>(s[i]);
        sums[0] = __builtin_fmaf(f, f, sums[0]);
        sums[1] = __builtin_fmaf(P::template get<j>(g[i]) * P::template get<j>(w[i]), f, sums[1]);
      });
    });
    // two places in turn: a wavefront may be a row ahead of another
    row_sums<WAVES>(sums, lds + turn * 2 * WAVES);
    turn ^= 1;
    const float r = inverse_rms(sums[0], d.H, a.eps);
    const float c = sums[1] * r / (float)d.H;   // mean(grad * w * n)
    static_for<VPT>([&](auto i) {
      const int v = i * (WAVES * kWave) + t;
      float o[N];
      static_for<N>([&](auto j) {
        const float n = P::template get<j>(s[i]) * r, gj = P::template get<j>(g[i]);
        dw[i][j] = __builtin_fmaf(gj, n, dw[i][j]);
        o[j] = r * __builtin_fmaf(gj, P::template get<j>(w[i]), -(n * c));
        if (a.grad_sum) o[j] += P::template get<j>(m[i]);
      });
      const row16_t out = pack<DT>(o);
      if (v < V) store_stream16(static_cast<row16_t*>(a.grad_x) + row * V + v, out);
    });
  }
  if (!a.grad_weight) return;
  // one part a block, also where it had no row: every part is read
  if constexpr (WAVES == 1) {
    __shared__ float others[kRows - 1][VPT * N][kWave];
    const int wave = threadIdx.x / kWave;
    if (wave > 0)
      static_for<VPT>([&](auto i) {
        static_for<N>([&](auto j) { others[wave - 1][i * N + j][t] = dw[i][j]; });
      });
    __syncthreads();
    if (wave > 0) return;
    static_for<kRows - 1>([&](auto w) {
      static_for<VPT>([&](auto i) {
        static_for<N>([&](auto j) { dw[i][j] += others[w][i * N + j][t]; });
      });
    });
  }
  static_for<VPT>([&](auto i) {
    const int v = i * (WAVES * kWave) + t;
    if (v < V) {
      float* to = a.partial + (int64_t)blockIdx.x * d.H + (int64_t)v * N;
      static_for<N / 4>([&](auto j) {
        reinterpret_cast<row16_t*>(to)[j] =
            row16_t{__float_as_uint(dw[i][4 * j]), __float_as_uint(dw[i][4 * j + 1]),
                    __float_as_uint(dw[i][4 * j + 2]), __float_as_uint(dw[i][4 * j + 3])};
      });
    }
  });
}

// The partial weight gradients added up, in an order that the sizes alone fix:
// a block has 16 columns, lanes of four, 256 rows at a time.
constexpr int kSumThreads = 1024, kSumCols = 16;
template <int DT>
__global__ void __launch_bounds__(kSumThreads)
    norm_weight_sum_kernel(const float* __restrict__ partial, int64_t rows, int64_t H,
                           void* __restrict__ grad_weight) {
  __shared__ f32x4 lds[kSumThreads / kWave][4];
  const int q = threadIdx.x % 4;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + q * 4;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (col < H)
    for (int64_t r = threadIdx.x / 4; r < rows; r += kSumThreads / 4)
      sum += *reinterpret_cast<const f32x4*>(partial + r * H + col);
  static_for<4>([&](auto i) {
    static_for<4>([&](auto c) { sum[c.value] += __shfl_xor(sum[c.value], 4 << i, kWave); });
  });
  if (lane_id() < 4) lds[threadIdx.x / kWave][q] = sum;
  __syncthreads();
  if (threadIdx.x < 4 && col < H) {
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
    static_for<kSumThreads / kWave>([&](auto w) { sum += lds[w][q]; });
    if constexpr (DT == EP_DTYPE_FP32) {
      *reinterpret_cast<row16_t*>(static_cast<float*>(grad_weight) + col) =
          row16_t{canon_f32(sum[0]), canon_f32(sum[1]), canon_f32(sum[2]), canon_f32(sum[3])};
    } else {
      uint16_t* to = static_cast<uint16_t*>(grad_weight) + col;
      static_for<4>([&](auto c) {
        to[c] = (uint16_t)(DT == EP_DTYPE_BF16 ? rne_bf16(sum[c.value]) : rne_f16(sum[c.value]));
      });
    }
  }
}

// Wavefronts to a row and vectors to a lane; V is at most EP_MAX_NORM_FEATURES
// values.
template <int DT, bool BWD, typename F>
hipError_t with_row(int64_t V, F&& f) {
  using std::integral_constant;
  if (V <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (V <= 128) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (V <= 256) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  if (V <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (V <= 1024) {
    // eight wavefronts, against four; 32768 rows of bf16 values with a residual, in 8
    // bits: 7168 values 271 us against 276, 8192 313 against 319, 6144 230 against 236,
    // but 5120 199 against 197 and 4224 183 against 166, where a lane's second vector
    // mostly lies past the row; 16 rows of 5120 4.3 against 5.2, of 7168 4.6 against
    // 5.6; fp32, 16384 rows of 4096, 141 against 142. Backward, where the weight's sums
    // are a lane's too, four
    if constexpr (!BWD) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  }
  if constexpr (DT == EP_DTYPE_FP32) {
    if (V > 2048) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  }
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

// Blocks of the backward pass, two a CU: each writes its part of the weight
// gradient. bf16 rows with a gradient of the sum, us with 512 blocks, and with 256,
// 1024 and 2048, whose parts are more bytes to write and read:
//   16384 x 4096    92   136  105  109       65536 x 1024     95   122  100  102
//   16384 x 7168   168   223  176  186       131072 x 512    110   192   98  102
//   8192 x 14336   179   173  193  223       262144 x 256    193   353  131  125
//   2048 x 4096     24    26   28   35       524288 x 64     351   671  217  201
// Narrow rows, one a wavefront, are few bytes in flight in 512 blocks: more would serve
// many of them better. fp32, 16384 x 4096: 183, 199, 191, 193.
constexpr int64_t kBwdBlocks = 512;
int64_t bwd_blocks(const Dims& d, int rows) {
  const int64_t blocks = (d.T + rows - 1) / rows;
  return blocks < 1 ? 1 : blocks < kBwdBlocks ? blocks : kBwdBlocks;
}

}  // namespace

hipError_t launch_rms_norm(const Dims& d, const NormArgs& a, hipStream_t stream) {
  return with_payload(d.dtype, [&](auto dt) {
    return with_row<decltype(dt)::value, false>(d.V, [&](auto waves, auto vpt) {
      constexpr int W = decltype(waves)::value;
      const int64_t blocks = (d.T + rows_of_block(W) - 1) / rows_of_block(W);
      // a grid has less than 2^32 threads in one direction: T < 2^31 rows of
      // 1024 threads may have more
      constexpr int64_t most = (int64_t)0xFFFFFFFF / threads_of_block(W);
      for (int64_t b0 = 0; b0 < blocks; b0 += most) {
        Dims part = d;
        NormArgs p = a;
        const int64_t r0 = b0 * rows_of_block(W), bytes = d.V * 16;
        const int64_t n = blocks - b0 < most ? blocks - b0 : most;
        part.T = d.T - r0;
        if (n * rows_of_block(W) < part.T) part.T = n * rows_of_block(W);
        auto at = [&](const void* q) {
          return q ? static_cast<const void*>(static_cast<const char*>(q) + r0 * bytes) : nullptr;
        };
        p.x = at(a.x);
        p.residual = at(a.residual);
        p.sum = const_cast<void*>(at(a.sum));
        p.out = const_cast<void*>(at(a.out));
        if (a.out_q) {
          p.out_q = a.out_q + r0 * d.H;
          p.out_scales = a.out_scales + r0 * EP_SCALE_COLUMNS(d.H);
        }
        rms_norm_kernel<decltype(dt)::value, W, decltype(vpt)::value>
            <<<dim3((uint32_t)n), dim3(threads_of_block(W)), 0, stream>>>(part, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    });
  });
}

int64_t norm_bwd_partials(const Dims& d) {
  int64_t n = 0;
  (void)with_payload(d.dtype, [&](auto dt) {
    return with_row<decltype(dt)::value, true>(d.V, [&](auto waves, auto) {
      n = bwd_blocks(d, rows_of_block(decltype(waves)::value));
      return hipSuccess;
    });
  });
  return n;
}

hipError_t launch_rms_norm_bwd(const Dims& d, const NormBwdArgs& a, hipStream_t stream) {
  return with_payload(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipError_t e = with_row<DT, true>(d.V, [&](auto waves, auto vpt) {
      constexpr int W = decltype(waves)::value;
      rms_norm_bwd_kernel<DT, W, decltype(vpt)::value>
          <<<dim3((uint32_t)bwd_blocks(d, rows_of_block(W))), dim3(threads_of_block(W)), 0,
             stream>>>(d, a);
      return hipGetLastError();
    });
    if (e != hipSuccess || !a.grad_weight) return e;
    norm_weight_sum_kernel<DT>
        <<<dim3((uint32_t)((d.H + kSumCols - 1) / kSumCols)), dim3(kSumThreads), 0, stream>>>(
            a.partial, norm_bwd_partials(d), d.H, a.grad_weight);
    return hipGetLastError();
  });
}

}  // namespace epmi
