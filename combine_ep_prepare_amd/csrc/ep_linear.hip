// ep_linear.hip -- products grouped by expert with ragged segments: each
// expert's weights applied to the live rows of its segment, and the two
// gradients of that product.

#include "ep_experts.h"

namespace epmi {

namespace {

// C = A B over one contraction index, one 64 x 64 tile of C per block step.
//   forward  C[r, n] = sum_h x[r, h] W[e][n, h]      rows r of expert e
//   dgrad    C[r, h] = sum_n g[r, n] W[e][n, h]
//   wgrad    C[n, h] = sum_r g[r, n] x[r, h]         for every expert e
enum Product { kForward, kRowGrad, kWeightGrad };

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <int DT, int P>
__global__ void __launch_bounds__(kThreads)
    grouped_product_kernel(Dims d, HandleView hv, const void* __restrict__ rows_a,
                           const void* __restrict__ b, void* __restrict__ c, int64_t N) {
  extern __shared__ int32_t tile_start[];
  __shared__ int32_t part[kThreads / kWave];
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t H = d.H;
  const int64_t cols = P == kForward ? N : H;
  const int64_t ct = (cols + kTile - 1) / kTile;
  const int64_t nt = (N + kTile - 1) / kTile;
  int64_t tiles;
  if constexpr (P == kWeightGrad) {
    tiles = (int64_t)d.E * nt * ct;
  } else {
    tiles = list_tiles<kThreads>(hv, d, kTile, tile_start, part) * ct;
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t rt = t / ct, c0 = (t - rt * ct) * kTile;
    const int e = P == kWeightGrad ? (int)(rt / nt)
                                   : expert_of_tile(tile_start, d.E, (int32_t)rt);
    const Segment s = segment_of(hv, d, e);
    const int64_t m0 = P == kWeightGrad ? (rt % nt) * kTile : (rt - tile_start[e]) * kTile;
    const int64_t M = P == kWeightGrad ? N : s.rows;
    const int64_t depth = P == kForward ? H : (P == kRowGrad ? N : s.rows);
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < depth; k0 += kStep) {
      for (int i = threadIdx.x; i < kStep * kTile; i += kThreads) {
        // the index along the operand's contiguous axis varies fastest
        int k, m;
        if (P == kWeightGrad) {
          k = i / kTile, m = i % kTile;
        } else {
          m = i / kStep, k = i % kStep;
        }
        float v = 0.f;
        if (k0 + k < depth && m0 + m < M) {
          v = P == kWeightGrad ? load_elem<DT>(rows_a, (s.row + k0 + k) * N + m0 + m)
                               : load_elem<DT>(rows_a, (s.row + m0 + m) * depth + k0 + k);
        }
        sa[k][m] = v;
        int n;
        if (P == kForward) {
          n = i / kStep, k = i % kStep;
        } else {
          k = i / kTile, n = i % kTile;
        }
        v = 0.f;
        if (k0 + k < depth && c0 + n < cols) {
          if (P == kForward) {
            v = load_elem<DT>(b, ((int64_t)e * N + c0 + n) * H + k0 + k);
          } else if (P == kRowGrad) {
            v = load_elem<DT>(b, ((int64_t)e * N + k0 + k) * H + c0 + n);
          } else {
            v = load_elem<DT>(b, (s.row + k0 + k) * H + c0 + n);
          }
        }
        sb[k][n] = v;
      }
      __syncthreads();
      for (int k = 0; k < kStep; ++k) {
        static_for<4>([&](auto i) {
          static_for<4>([&](auto j) {
            acc[i][j] = __builtin_fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
          });
        });
      }
      __syncthreads();
    }
    static_for<4>([&](auto i) {
      static_for<4>([&](auto j) {
        const int64_t m = m0 + ty * 4 + i, n = c0 + tx * 4 + j;
        if (m < M && n < cols) {
          const int64_t r = P == kWeightGrad ? (int64_t)e * N + m : s.row + m;
          store_elem<DT>(c, r * cols + n, acc[i][j]);
        }
      });
    });
  }
  if constexpr (P != kWeightGrad)
    write_zero_rows(hh, hv, d, c, cols * (DT == EP_DTYPE_FP32 ? 4 : 2) / 16);
}

template <int P>
hipError_t launch_product(const Dims& d, const HandleView& hv, const void* a, const void* b,
                          void* c, int64_t N, int num_cus, hipStream_t stream) {
  const size_t lds = P == kWeightGrad ? 0 : sizeof(int32_t) * (size_t)(d.E + 1);
  return with_payload(d.dtype, [&](auto dt) {
    grouped_product_kernel<decltype(dt)::value, P>
        <<<dim3(num_cus * 4), dim3(kThreads), lds, stream>>>(d, hv, a, b, c, N);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_grouped_linear(const Dims& d, const HandleView& hv, const void* x,
                                 const void* weight, void* out, int64_t N, int num_cus,
                                 hipStream_t stream) {
  return launch_product<kForward>(d, hv, x, weight, out, N, num_cus, stream);
}

hipError_t launch_grouped_linear_bwd(const Dims& d, const HandleView& hv, const void* grad,
                                     const void* x, const void* weight, void* grad_x,
                                     void* grad_weight, int64_t N, int num_cus,
                                     hipStream_t stream) {
  if (grad_x) {
    const hipError_t e =
        launch_product<kRowGrad>(d, hv, grad, weight, grad_x, N, num_cus, stream);
    if (e != hipSuccess) return e;
  }
  if (grad_weight)
    return launch_product<kWeightGrad>(d, hv, grad, x, grad_weight, N, num_cus, stream);
  return hipSuccess;
}

}  // namespace epmi
