// ep_choice.h -- which kernel and tile an expert product runs with, from what
// the host knows: the layout, the feature counts and the CU count.
#pragma once

#include "ep.h"
#include "ep_internal.h"

namespace epmi {

enum Product { kForward, kRowGrad, kWeightGrad };

enum class Kernel {
  kFewRows,   // ep_decode.hip
  // ep_linear.hip, by the tile; Once: what one tile alone uses passes by the caches
  kTile256,
  kTile256Once,
  kTile128,
  kTile128Once,
  kTile64,
};

// The most rows that all experts together can have: a route has one at most, and
// none past the capacity. On a rank that holds a few of the experts most routes
// are masked, and the capacity is what tells.
inline int64_t most_rows(const Dims& d) {
  const int64_t routes = d.T * d.K;
  return routes < d.cap ? routes : d.cap;
}

// The rules go by rows per expert, were the most rows spread evenly. Measured in
// bf16 at 128 experts, 2048 inputs and 1536 outputs, no route masked, the capacity
// no less than the routes, unless another size is named; a rank's 32 of 256
// experts (7168 inputs, 4096 outputs, a capacity a quarter above its rows) has its
// borders at about the same rows.
inline Kernel kernel_of(Product p, const Dims& d, int64_t N, int num_cus) {
  const bool bits16 = d.dtype != EP_DTYPE_FP32;
  const int64_t per_expert = most_rows(d) / d.E;
  // of a segment's tiles: rows, or N in the weight gradient
  const int64_t rows = p == kWeightGrad ? N : per_expert;
  const int64_t cols = p == kForward ? N : d.H;
  if (bits16) {
    // up to 12 rows: 8 rows 135 us against 144 with the tiles below, one row 90
    // against 103; 16 rows 193 against 152 (many experts then have more rows
    // than the 16 of its pass)
    if (p == kForward && rows <= 12) return Kernel::kFewRows;
    // 256 x 256 tiles, if they fill the CUs. Forward from 105 rows, where many
    // experts have a second tile of 128: 104 rows 214 us against 205, 112 rows 213
    // against 225. Row gradient, whose weights come in by lines of k, from 33: 32
    // rows 156 against 155, 40 rows 159 against 161, 128 rows 177 against 218; with
    // less than two tiles a CU as forward (32 experts of 94 rows: 47 against 43).
    // Rows that fill two tiles of 128 leave the larger ahead on three quarters of
    // the CUs too (32 experts of 128 rows, forward: 64 against 78).
    const int64_t tiles = (rows + 255) / 256 * ((cols + 255) / 256) * d.E;
    const int64_t from = p == kWeightGrad ? 129 : p == kRowGrad && tiles >= 2 * num_cus ? 33 : 105;
    const int64_t fill = p != kWeightGrad && rows > 128 ? num_cus * 3 / 4 : num_cus;
    if (rows >= from && cols > 128 && tiles >= fill) {
      // weight gradients are stored past the caches up to 768 rows an expert,
      // where their bytes count more than the products: 1 row 192 us against
      // 204, 256 rows 370 against 400, 768 rows 660 against 672, but 1027 rows
      // (7168 inputs, 4096 outputs) 1828 against 1820 and 4096 2970 against 2918
      return p == kWeightGrad && per_expert <= 768 ? Kernel::kTile256Once : Kernel::kTile256;
    }
  }
  // 64 x 64 tiles where larger ones would leave CUs without work (one expert of
  // 256 rows, 4096 x 4096: 27 us against 44; fp32's weight gradient of five of
  // 6150 rows, 224 x 320: 121 against 413). fp32 is bound by its matrix
  // instructions, not by loads, and gains up to four of the larger a CU.
  const int64_t tiles = (rows + 127) / 128 * ((cols + 127) / 128) * d.E;
  if (tiles < (bits16 ? 1 : 4) * num_cus) return Kernel::kTile64;
  // weights past the caches up to 104 rows, where most experts have one row
  // tile: 16 rows 152 us against 166, 64 rows 173 against 178, 104 rows 205 against
  // 208; at 128 rows half of them have two, 265 against 231
  if (bits16 && p != kWeightGrad && rows <= 104) return Kernel::kTile128Once;
  return Kernel::kTile128;
}

}  // namespace epmi
