// ep_device.h -- device helpers shared by the kernel files: the handle check,
// the zero rows of an expert-major output, payload types and their rounding,
// and the streaming store.
#pragma once

#include <hip/hip_runtime.h>

#include <utility>

#include "ep.h"
#include "ep_internal.h"

namespace epmi {

namespace {

// Compile-time loop: f(std::integral_constant<int, i>) for i in [0, N). Keeps
// every index of the small per-lane register arrays a constant, so they stay
// in VGPRs instead of being demoted to LDS or scratch.
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & (kWave - 1); }

__device__ __forceinline__ uint64_t wave_ballot(bool p) {
  return static_cast<uint64_t>(__ballot(p));
}

// 16 bytes per lane (8 bf16 or fp16, or 4 fp32); a wavefront moves 1 KiB per
// instruction.
typedef uint32_t row16_t __attribute__((ext_vector_type(4)));

// The whole header is copied in one go and then tested without
// short-circuits, so it costs one round trip instead of one per field.
__device__ __forceinline__ bool handle_matches(const HandleHeader& hh, const Dims& d) {
  return (hh.magic == kHandleMagic) & (hh.num_tokens == d.T) & (hh.topk == d.K) &
         (hh.num_experts == d.E) & (hh.alignment == d.A) & (hh.recv_capacity == d.cap) &
         (hh.total >= 0) & (hh.pads_live >= 0);
}

// Rows a payload op writes as zeros, in this order: the live pad rows
// (pad_rows[0, npads), ascending) when pads are filled, then the rows past the
// live total (live .. cap-1) when the tail is zeroed.
struct ZeroRows {
  int64_t npads;  // pad rows among them
  int64_t n;      // all of them
  int64_t live;   // min(total, cap): the first tail row
};

__device__ __forceinline__ ZeroRows zero_rows_of(const HandleHeader& hh, const Dims& d) {
  ZeroRows z;
  z.live = (int64_t)hh.total < d.cap ? (int64_t)hh.total : d.cap;
  z.npads = d.fill_pads ? (int64_t)hh.pads_live : 0;
  z.n = z.npads + (d.zero_tail ? d.cap - z.live : 0);
  return z;
}

__device__ __forceinline__ int64_t zero_row(const ZeroRows& z,
                                            const int32_t* __restrict__ pad_rows, int64_t i) {
  return i < z.npads ? (int64_t)pad_rows[i] : z.live + (i - z.npads);
}

// fp32 -> bf16 bits, round to nearest even; any NaN -> 0x7FC0. Adding
// 0x7FFF plus the lowest kept bit carries into the kept half exactly when the
// discarded half is above one half ulp, or equal to it with an odd kept half.
__device__ __forceinline__ uint32_t rne_bf16(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Streaming stores write through the XCD's L2: non-temporal at system scope
// (cache-policy bits sc0 sc1 nt of the CDNA3/CDNA4 vector memory
// instructions). A plain non-temporal store (nt alone) leaves its lines
// dirty in the L2 until they are evicted, where they push out rows that are
// still to be read; measured on the MI355X, the dsv3 dispatch by run entries
// takes 118 µs with the write-through form against 125 µs (its token rows
// are then read from HBM once), and no op is slower. The compiler emits no
// such store from C++, so it is written out. A store of more than 64 bits of
// data needs two wait states on the gfx940 family (gfx950 included) before a
// VALU instruction may overwrite its data registers, and the compiler inserts
// none after an asm statement: `s_nop 1` gives both. With one (`s_nop 0`) a
// GPU test saw the next loop step's index stored in place of the data.
__device__ __forceinline__ void store_stream16(row16_t* p, row16_t v) {
  asm volatile("global_store_dwordx4 %0, %1, off sc0 sc1 nt\n\ts_nop 1" ::"v"(p), "v"(v)
               : "memory");
}

// fp32 -> fp16 bits: the hardware conversion rounds to nearest even and keeps
// fp16 subnormals; any NaN -> 0x7E00. The fp32 value is first made opaque to
// the compiler: otherwise it may fold the multiply or fused multiply-add that
// produced it into one mixed-precision instruction (v_fma_mixlo_f16) that
// rounds the exact result straight to fp16, skipping the fp32 rounding the
// result is defined by.
__device__ __forceinline__ uint32_t rne_f16(float f) {
  asm("" : "+v"(f));
  if (__builtin_isnan(f)) return 0x7E00u;
  return __builtin_bit_cast(unsigned short, static_cast<_Float16>(f));
}

__device__ __forceinline__ float f16_to_f32(uint32_t bits16) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(bits16)));
}

// fp32 result bits: the value itself, any NaN -> 0x7FC00000.
__device__ __forceinline__ uint32_t canon_f32(float f) {
  const uint32_t u = __float_as_uint(f);
  return ((u & 0x7FFFFFFFu) > 0x7F800000u) ? 0x7FC00000u : u;
}

// Payload element types. A 16-byte vector holds N elements; get<I> widens
// element I exactly to fp32 and pack rounds N fp32 values once to the type.
template <int DT>
struct Payload;

template <>
struct Payload<EP_DTYPE_BF16> {
  static constexpr int N = 8;
  template <int I>
  __device__ static __forceinline__ float get(const row16_t& v) {
    return (I & 1) ? bf16_hi(v[I >> 1]) : bf16_lo(v[I >> 1]);
  }
  __device__ static __forceinline__ row16_t pack(const float (&a)[N]) {
    row16_t o;
    static_for<4>([&](auto q) {
      constexpr int i = q;
      o[i] = rne_bf16(a[2 * i]) | (rne_bf16(a[2 * i + 1]) << 16);
    });
    return o;
  }
};

template <>
struct Payload<EP_DTYPE_FP16> {
  static constexpr int N = 8;
  template <int I>
  __device__ static __forceinline__ float get(const row16_t& v) {
    return f16_to_f32((I & 1) ? (v[I >> 1] >> 16) : (v[I >> 1] & 0xFFFFu));
  }
  __device__ static __forceinline__ row16_t pack(const float (&a)[N]) {
    row16_t o;
    static_for<4>([&](auto q) {
      constexpr int i = q;
      o[i] = rne_f16(a[2 * i]) | (rne_f16(a[2 * i + 1]) << 16);
    });
    return o;
  }
};

template <>
struct Payload<EP_DTYPE_FP32> {
  static constexpr int N = 4;
  template <int I>
  __device__ static __forceinline__ float get(const row16_t& v) {
    return __uint_as_float(v[I]);
  }
  __device__ static __forceinline__ row16_t pack(const float (&a)[N]) {
    row16_t o;
    static_for<4>([&](auto q) {
      constexpr int i = q;
      o[i] = canon_f32(a[i]);
    });
    return o;
  }
};

}  // namespace

}  // namespace epmi
