// ep_linear.hip -- products grouped by expert with ragged segments: each
// expert's weights applied to the live rows of its segment, and the two
// gradients of that product.
//
//   forward  C[r, n] = sum_h x[r, h] W[e][n, h]      rows r of expert e
//   dgrad    C[r, h] = sum_n g[r, n] W[e][n, h]
//   wgrad    C[n, h] = sum_r g[r, n] x[r, h]         for every expert e
//
// Each is C = A B over one contraction index k. An operand is K-major when k
// is its contiguous axis (x and W forward, g in dgrad), else MN-major (W in
// dgrad, both operands in wgrad).

#include "ep_experts.h"

namespace epmi {

namespace {

enum Product { kForward, kRowGrad, kWeightGrad };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

typedef __attribute__((address_space(3))) char lds_char;

// One fragment of 16 rows (or columns) of an operand for a lane: 16 bytes, 8
// (16-bit types) or 4 (fp32) values of k. The order of k inside a fragment
// is the same for both operands, which is all that the sum needs.
template <int DT>
__device__ __forceinline__ void mma(f32x4& acc, row16_t n, row16_t m) {
  if constexpr (DT == EP_DTYPE_BF16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, n), __builtin_bit_cast(bf16x8, m), acc, 0, 0, 0);
  } else if constexpr (DT == EP_DTYPE_FP16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(
        __builtin_bit_cast(f16x8, n), __builtin_bit_cast(f16x8, m), acc, 0, 0, 0);
  } else {
    static_for<4>([&](auto t) {
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(n[t.value]), __uint_as_float(m[t.value]),
                                                 acc, 0, 0, 0);
    });
  }
}

// A buffer resource over `bytes` bytes at p: a lane whose offset lies at or
// past them reads zeros.
__device__ __forceinline__ row16_t buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return row16_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// An offset past every buffer of a tile (256 rows of EP_MAX_FEATURES values).
constexpr uint32_t kOutside = 0x40000000u;

// 16 bytes per lane from a buffer straight into LDS: lane l's bytes land at
// lds + 16 l. Written out because the compiler makes every later LDS read
// wait for such loads, also those of the other half of a double buffer; the
// wait is in sync_stage below. Nothing else here lives in m0: the compiler
// sets it right before each of its own uses.
__device__ __forceinline__ void load_to_lds(row16_t buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(offset), "s"(buffer)
               : "memory");
}

// Every load of this wavefront has landed and every LDS read is done, for
// all wavefronts of the block.
__device__ __forceinline__ void sync_stage() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One operand's tile of a step: R rows (or columns) by 128 bytes of k, i.e.
// 64 values of a 16-bit type or 32 of fp32, in LDS as R * 128 bytes.
//
// K-major: a row is 128 bytes of k, its 16-byte chunk c at slot c ^ (row & 7),
// so that the 16 rows a fragment read touches spread over the banks. A lane
// reads 16 bytes of one row.
// MN-major: a line of k holds R values in granules of 16; granule g sits at
// g ^ f(k). A fragment read takes 16-bit values by the transposing LDS read
// (16 lanes read 4 lines of 16 values, each lane receives one column of 4), and
// fp32 one value a lane; f spreads the lines that one read touches.
// The swizzles are applied to the global side of the loads, whose LDS side is
// linear.
template <int DT, bool KMAJOR, int R>
struct Operand {
  static constexpr int kSize = DT == EP_DTYPE_FP32 ? 4 : 2;
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = kBytes / 1024;           // wavefront loads of a tile
  static constexpr int kDepth = 128 / kSize;             // values of k
  static constexpr int kLine = R * kSize;                // MN-major: bytes of a line
  static constexpr int kGranules = R / 16;

  __device__ static __forceinline__ int swizzle(int k) {
    const int f = kSize == 2 ? (k & 3) | ((k >> 1) & 12) : (k >> 2) & 3;
    return f & (kGranules - 1);
  }

  // This lane's offset, in the tile's source, of wavefront load i: K-major
  // relative to (row 0, k 0) of the tile with rows of `stride` bytes, without
  // the k of the step; MN-major relative to (k 0, column 0) of the step's lines
  // of `stride` bytes, kOutside for columns at or past `cols`.
  __device__ static __forceinline__ uint32_t source(int i, uint32_t stride, int64_t cols) {
    const int lane = lane_id();
    if constexpr (KMAJOR) {
      return (uint32_t)(i * 8 + lane / 8) * stride;
    } else {
      const int at = i * 1024 + lane * 16;
      const int k = at / kLine, slot = (at % kLine) / 16;
      const int g = (slot / kSize) ^ swizzle(k);
      const int chunk = g * kSize + slot % kSize;
      return chunk * (16 / kSize) < cols ? (uint32_t)k * stride + chunk * 16 : kOutside;
    }
  }
  // K-major: the first value of k, in the step, of this lane's chunk.
  __device__ static __forceinline__ int chunk_k() {
    const int lane = lane_id();
    return ((lane & 7) ^ (lane / 8)) * (16 / kSize);
  }

  // LDS offset of this lane's part of the fragment that starts at row (or
  // column) `first`, for half `half` of the step's k.
  __device__ static __forceinline__ uint32_t fragment(int first, int half) {
    const int lane = lane_id(), i = lane & 15, q = lane >> 4;
    if constexpr (KMAJOR) {
      return (first + i) * 128 + (((half * 4 + q) ^ (i & 7)) << 4);
    } else if constexpr (kSize == 2) {
      const int k = half * 32 + q * 8 + (i >> 2);
      return k * kLine + (((first >> 4) ^ swizzle(k)) << 5) + (i & 3) * 8;
    } else {
      const int k = half * 16 + q * 4;
      return k * kLine + (((first >> 4) ^ swizzle(k)) << 6) + i * 4;
    }
  }
  __device__ static __forceinline__ row16_t read(uint32_t at) {
    if constexpr (KMAJOR) {
      return *reinterpret_cast<__attribute__((address_space(3))) row16_t*>((lds_char*)(uintptr_t)at);
    } else if constexpr (kSize == 2) {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)at);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)(at + 4 * kLine));
      return __builtin_bit_cast(row16_t, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    } else {
      row16_t v;
      static_for<4>([&](auto t) {
        v[t.value] = *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(
            (lds_char*)(uintptr_t)(at + t * kLine));
      });
      return v;
    }
  }
};

// Four results of a row, rounded and stored.
template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, f32x4 v) {
  if constexpr (DT == EP_DTYPE_FP32) {
    *reinterpret_cast<row16_t*>(static_cast<float*>(p) + i) =
        row16_t{canon_f32(v[0]), canon_f32(v[1]), canon_f32(v[2]), canon_f32(v[3])};
  } else if constexpr (DT == EP_DTYPE_BF16) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) = u32x2{
        rne_bf16(v[0]) | (rne_bf16(v[1]) << 16), rne_bf16(v[2]) | (rne_bf16(v[3]) << 16)};
  } else {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) = u32x2{
        rne_f16(v[0]) | (rne_f16(v[1]) << 16), rne_f16(v[2]) | (rne_f16(v[3]) << 16)};
  }
}

// Row tiles of an expert whose column tiles run together: with the columns
// dealt after them, the tiles in flight on an XCD share both operands.
constexpr int kGroup = 8;
// Weight-gradient tiles that go to one XCD together: one for each of its CUs.
constexpr int kChunk = 32;


// One block step is a BM x BN tile of C: WM x WN wavefronts, each with a part
// of (BM / WM) x (BN / WN) in registers as 16 x 16 blocks. Steps of 128 bytes
// of k go through two LDS buffers: the loads of a step are in flight while
// the one before is multiplied, one barrier a step.
template <int DT, int P, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(WM* WN* kWave)
    grouped_product_kernel(Dims d, HandleView hv, const void* __restrict__ a,
                           const void* __restrict__ b, void* __restrict__ c, int64_t N) {
  using A = Operand<DT, P != kWeightGrad, BM>;
  using B = Operand<DT, P == kForward, BN>;
  constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
  constexpr int kStage = A::kBytes + B::kBytes;
  constexpr int AL = A::kLoads / kWaves, BL = B::kLoads / kWaves;
  static_assert(AL * kWaves == A::kLoads && BL * kWaves == B::kLoads, "whole loads");
  extern __shared__ __align__(1024) char lds[];
  int32_t* tile_start = reinterpret_cast<int32_t*>(lds + 2 * kStage);
  int32_t* part = tile_start + d.E + 1;

  const HandleHeader hh = *hv.header;
  if (!handle_matches(hh, d)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&hv.header->status, EP_STATUS_LAYOUT);
    return;
  }
  const int64_t H = d.H;
  const int64_t cols = P == kForward ? N : H;
  const int32_t ct = (int32_t)((cols + BN - 1) / BN);
  const int32_t nt = (int32_t)((N + BM - 1) / BM);  // wgrad: row tiles of every expert
  int64_t tiles;
  if constexpr (P == kWeightGrad) {
    tiles = (int64_t)d.E * nt * ct;
  } else {
    tiles = (int64_t)list_tiles<kThreads>(hv, d, BM, tile_start, part) * ct;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int lane = lane_id();
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_char*)lds;
  // Blocks are dealt round-robin to the XCDs: chunks of consecutive tiles go
  // to one XCD each in turn. A grid of fewer blocks than tiles (not wgrad)
  // makes a chunk of what an XCD works on at once.
  const int64_t slots = P == kWeightGrad ? kChunk : gridDim.x / kRunXcds;
  const int64_t xcd = blockIdx.x % kRunXcds, slot = blockIdx.x / kRunXcds;
  int64_t t = ((slot / slots) * kRunXcds + xcd) * slots + slot % slots;
  for (; t < tiles; t += P == kWeightGrad ? tiles : (int64_t)gridDim.x) {
    // tile t: expert e, row tile mi, column tile ni
    int e;
    int64_t first;
    int32_t rts;
    if constexpr (P == kWeightGrad) {
      e = (int)(t / ((int64_t)nt * ct));
      first = (int64_t)e * nt * ct;
      rts = nt;
    } else {
      e = expert_of_tile(tile_start, d.E, (int32_t)(t / ct));
      e = __builtin_amdgcn_readfirstlane(e);
      first = (int64_t)tile_start[e] * ct;
      rts = tile_start[e + 1] - tile_start[e];
    }
    const int64_t in_e = t - first;
    const int32_t group = (int32_t)(in_e / ((int64_t)kGroup * ct));
    const int32_t in_g = (int32_t)(in_e - (int64_t)group * kGroup * ct);
    const int32_t gm = rts - group * kGroup < kGroup ? rts - group * kGroup : kGroup;
    const int64_t m0 = __builtin_amdgcn_readfirstlane((group * kGroup + in_g % gm) * BM);
    const int64_t n0 = __builtin_amdgcn_readfirstlane((in_g / gm) * BN);
    const Segment s = segment_of(hv, d, e);
    const int64_t M = P == kWeightGrad ? N : s.rows;
    const int32_t depth = (int32_t)(P == kForward ? H : (P == kRowGrad ? N : s.rows));
    const int32_t mrows = (int32_t)(M - m0 < BM ? M - m0 : BM);
    const int32_t ncols = (int32_t)(cols - n0 < BN ? cols - n0 : BN);
    constexpr int kSize = A::kSize;

    // sources of the two operands and their row (line) strides in bytes
    const uint32_t a_stride = (uint32_t)((P == kForward ? H : N) * kSize);
    const uint32_t b_stride = (uint32_t)(H * kSize);
    const char* a_src = static_cast<const char*>(a);
    const char* b_src = static_cast<const char*>(b);
    if constexpr (P == kWeightGrad) {
      a_src += s.row * a_stride + m0 * kSize;
      b_src += s.row * b_stride + n0 * kSize;
    } else {
      a_src += (s.row + m0) * a_stride;
      b_src += (int64_t)e * N * b_stride + (P == kForward ? n0 * b_stride : n0 * kSize);
    }
    const int steps = (depth + A::kDepth - 1) / A::kDepth;
    uint32_t a_off[AL], b_off[BL];
    static_for<AL>([&](auto i) {
      a_off[i] = A::source(wave * AL + i, a_stride, mrows);
    });
    static_for<BL>([&](auto i) {
      b_off[i] = B::source(wave * BL + i, b_stride, ncols);
    });

    auto load_stage = [&](int step, int buf) {
      const int32_t k0 = step * A::kDepth;
      const int32_t left = depth - k0;
      const int32_t lines = left < A::kDepth ? left : A::kDepth;
      const uint32_t to = lds_base + buf * kStage;
      const int chunk = A::chunk_k();
      const uint32_t ko = chunk < left ? (uint32_t)(k0 + chunk) * kSize : kOutside;
      if constexpr (P != kWeightGrad) {
        const row16_t r = buffer_of(a_src, (uint32_t)mrows * a_stride);
        static_for<AL>([&](auto i) {
          load_to_lds(r, a_off[i] + ko, to + (wave * AL + i) * 1024);
        });
      } else {
        const row16_t r = buffer_of(a_src + (int64_t)k0 * a_stride, (uint32_t)lines * a_stride);
        static_for<AL>([&](auto i) {
          load_to_lds(r, a_off[i], to + (wave * AL + i) * 1024);
        });
      }
      if constexpr (P == kForward) {
        const row16_t r = buffer_of(b_src, (uint32_t)ncols * b_stride);
        static_for<BL>([&](auto i) {
          load_to_lds(r, b_off[i] + ko, to + A::kBytes + (wave * BL + i) * 1024);
        });
      } else {
        const row16_t r = buffer_of(b_src + (int64_t)k0 * b_stride, (uint32_t)lines * b_stride);
        static_for<BL>([&](auto i) {
          load_to_lds(r, b_off[i], to + A::kBytes + (wave * BL + i) * 1024);
        });
      }
    };

    f32x4 acc[MF][NF];
    static_for<MF>([&](auto i) {
      static_for<NF>([&](auto j) { acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    });
    const bool busy = wm * (BM / WM) < mrows && wn * (BN / WN) < ncols;
    sync_stage();  // the last tile's reads are done
    if (steps > 0) load_stage(0, 0);
    for (int k = 0; k < steps; ++k) {
      sync_stage();
      if (k + 1 < steps) load_stage(k + 1, (k + 1) & 1);
      if (busy) {
        const uint32_t at = lds_base + (k & 1) * kStage;
        static_for<2>([&](auto half) {
          row16_t mf[MF], nf[NF];
          static_for<NF>([&](auto j) {
            nf[j] = B::read(at + A::kBytes + B::fragment(wn * (BN / WN) + j * 16, half));
          });
          static_for<MF>([&](auto i) {
            mf[i] = A::read(at + A::fragment(wm * (BM / WM) + i * 16, half));
          });
          static_for<MF>([&](auto i) {
            static_for<NF>([&](auto j) { mma<DT>(acc[i][j], nf[j], mf[i]); });
          });
        });
      }
    }
    // a lane holds four consecutive columns of one row of each 16 x 16 block
    if (busy) {
      static_for<MF>([&](auto i) {
        const int32_t m = wm * (BM / WM) + i * 16 + (lane & 15);
        if (m < mrows) {
          const int64_t r = P == kWeightGrad ? (int64_t)e * N + m0 + m : s.row + m0 + m;
          static_for<NF>([&](auto j) {
            const int32_t n = wn * (BN / WN) + j * 16 + (lane >> 4) * 4;
            if (n < ncols) store4<DT>(c, r * cols + n0 + n, acc[i][j]);
          });
        }
      });
    }
  }
  if constexpr (P != kWeightGrad) {
    write_zero_rows(hh, hv, d, c, cols * A::kSize / 16);
  }
}

template <int DT, int P, int BM, int BN, int WM, int WN>
hipError_t launch_tiles(const Dims& d, const HandleView& hv, const void* a, const void* b,
                        void* c, int64_t N, int num_cus, int per_cu, hipStream_t stream) {
  auto* kernel = grouped_product_kernel<DT, P, BM, BN, WM, WN>;
  const int64_t cols = P == kForward ? N : d.H;
  const int64_t ct = (cols + BN - 1) / BN;
  // the most row tiles that the routing may need: every route's row, and one
  // part tile an expert
  const int64_t routes = d.T * d.K < d.cap ? d.T * d.K : d.cap;
  int64_t blocks;
  if (P == kWeightGrad) {
    blocks = (int64_t)d.E * ((N + BM - 1) / BM) * ct;
  } else {
    blocks = (routes / BM + (d.E < routes ? d.E : routes)) * ct;
    const int64_t most = (int64_t)num_cus * per_cu;
    if (blocks > most) blocks = most;
  }
  const int64_t unit = P == kWeightGrad ? kRunXcds * kChunk : kRunXcds;
  blocks = (blocks + unit - 1) / unit * unit;
  if (blocks < unit) blocks = unit;
  if (blocks > 0x7FFFFF00) return hipErrorInvalidConfiguration;
  const size_t lds = 2 * (size_t)(BM + BN) * 128 + sizeof(int32_t) * (size_t)(d.E + 1 + 16);
  kernel<<<dim3((uint32_t)blocks), dim3(WM * WN * kWave), lds, stream>>>(d, hv, a, b, c, N);
  return hipGetLastError();
}

template <int P>
hipError_t launch_product(const Dims& d, const HandleView& hv, const void* a, const void* b,
                          void* c, int64_t N, int num_cus, hipStream_t stream) {
  return with_payload(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const int64_t rows = P == kWeightGrad ? N : d.T * d.K / d.E;
    const int64_t cols = P == kForward ? N : d.H;
    if constexpr (DT != EP_DTYPE_FP32) {
      if (P == kForward && rows <= 16) return launch_grouped_few(d, hv, a, b, c, N, num_cus, stream);
      if (rows > 128 && cols > 128)
        return launch_tiles<DT, P, 256, 256, 2, 4>(d, hv, a, b, c, N, num_cus, 1, stream);
    }
    return launch_tiles<DT, P, 128, 128, 2, 2>(d, hv, a, b, c, N, num_cus, 2, stream);
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
