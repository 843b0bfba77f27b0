// ep_tiles.h -- what the tiled products have in common (ep_linear.hip,
// ep_scaled.hip): loads from global memory straight into LDS, the layout of an
// operand's tile there, and the joining of results.
#pragma once

#include "ep_experts.h"
#include "ep_matrix.h"

namespace epmi {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

typedef __attribute__((address_space(3))) char lds_char;

// A buffer resource over `bytes` bytes at p: a lane whose offset lies at or
// past them reads zeros.
__device__ __forceinline__ row16_t buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  // the same in every lane; the load wants it in scalar registers
  return row16_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xFFFFu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

// An offset past every buffer of a tile (256 rows of EP_MAX_FEATURES values).
constexpr uint32_t kOutside = 0x40000000u;

// 16 bytes per lane from a buffer straight into LDS: lane l's bytes land at
// lds + at + 16 l. Written out because the compiler makes every later LDS read wait
// for such loads, also those of the other half of a double buffer; the wait is in
// sync_loads below. The place goes through m0, which is reserved in the compiler
// and which nothing else here uses.
// The load needs five wait states behind a vector instruction that wrote one of
// the buffer's scalar registers (a register brought back from a lane, say, which
// may come right before it), and one behind the write of m0. The compiler counts
// neither for an asm statement, so it holds both. They cost the large products
// between 1 and 2% (backward of 8 experts of 4096 rows, 14336 x 4096: 6050 us without
// and 6170 with them); two loads a statement, which share one wait, cost 3%.
// ONCE: the bytes are read by one tile only and need not stay in the caches.
template <bool ONCE, int AT>
__device__ __forceinline__ void load_to_lds(row16_t buffer, uint32_t offset, uint32_t lds) {
  if constexpr (ONCE) {
    asm volatile(
        "s_add_u32 m0, %2, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" ::"v"(
            offset),
        "s"(buffer), "s"(lds), "n"(AT)
        : "memory", "scc");
  } else {
    asm volatile(
        "s_add_u32 m0, %2, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset),
        "s"(buffer), "s"(lds), "n"(AT)
        : "memory", "scc");
  }
}

// For all wavefronts of the block: every LDS read is done, and every load
// to LDS but the LATEST youngest of each has landed.
template <int LATEST>
__device__ __forceinline__ void sync_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATEST) : "memory");
}

// One operand's tile of a step: R rows (or columns) by 128 bytes of k, i.e.
// 128 values in 8 bits (K-major only), 64 of a 16-bit type or 32 of fp32, in LDS
// as R * 128 bytes.
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
constexpr int kBytes8 = -1;   // in place of a payload type: values in 8 bits
template <int DT, bool KMAJOR, int R, int EVERY>
struct Operand {
  static constexpr int kSize = DT == kBytes8 ? 1 : DT == EP_DTYPE_FP32 ? 4 : 2;
  static_assert(kSize > 1 || KMAJOR, "8 bits: K-major");
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
      return (uint32_t)(i * 8 + lane / 8) * stride + chunk_k() * kSize;
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

  // Fragment f (16 rows or columns from first + 16 f EVERY) of half h of the
  // step's k, for this lane: at(first, K-major ? h : f) plus a constant.
  static constexpr int addresses(int fragments) { return KMAJOR ? 2 : fragments; }
  __device__ static __forceinline__ uint32_t at(int first, int index) {
    const int lane = lane_id(), i = lane & 15, q = lane >> 4;
    if constexpr (KMAJOR) {
      return (first + i) * 128 + (((index * 4 + q) ^ (i & 7)) << 4);
    } else {
      const int k = kSize == 2 ? q * 8 + (i >> 2) : q * 4;
      const int g = ((first >> 4) + index * EVERY) ^ swizzle(k);
      return k * kLine + g * (16 * kSize) + (kSize == 2 ? (i & 3) * 8 : i * 4);
    }
  }
  template <int F, int HALF>
  __device__ static __forceinline__ row16_t read(uint32_t base) {
    const lds_char* p = (const lds_char*)(uintptr_t)base;
    if constexpr (KMAJOR) {
      return *reinterpret_cast<const __attribute__((address_space(3))) row16_t*>(p + F * EVERY * 2048);
    } else if constexpr (kSize == 2) {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      constexpr int kHalf = HALF * 32 * kLine;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + kHalf));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + kHalf + 4 * kLine));
      return __builtin_bit_cast(row16_t,
                                s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    } else {
      row16_t v;
      static_for<4>([&](auto t) {
        v[t.value] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(
            p + (HALF * 16 + t.value) * kLine);
      });
      return v;
    }
  }
};

// A lane of quarter q holds columns 4 q to 4 q + 3 of two neighbouring blocks
// of 16, and gets columns 8 q to 8 q + 7 of the 32: stores of 16 bytes, 64 to a
// row, in place of 8 and 32. Lanes trade with their like of the other quarters,
// which hold the same row. The weight gradient of 128 experts (2048 x 1536, 65536
// uneven rows) went from 688 to 623 us by it, of one row each from 272 to 203.
__device__ __forceinline__ row16_t join_blocks(u32x2 a, u32x2 b) {
  const auto lo = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  const auto l = __builtin_amdgcn_permlane16_swap(lo[0], lo[1], false, false);
  const auto h = __builtin_amdgcn_permlane16_swap(hi[0], hi[1], false, false);
  return row16_t{l[0], h[0], l[1], h[1]};
}

}  // namespace

}  // namespace epmi
