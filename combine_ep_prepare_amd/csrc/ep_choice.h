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
  // ep_scaled.hip alone: tiles with a ring of buffers
  kRing64,
  kRing128,
  kRing64x128,
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

// The same for the product of 8-bit operands (ep_scaled.hip), measured in bf16 at
// 128 experts, 2048 inputs and 1536 outputs unless another size is named.
inline Kernel scaled_kernel_of(const Dims& d, int64_t N, int num_cus) {
  const int64_t rows = most_rows(d) / d.E;
  // up to 6 rows: 2 rows 57 us against 62 with the tiles below, 6 rows 66 against 65;
  // 8 rows 67 against 64. One expert's few tiles leave most CUs without work, so that
  // up to 32 rows those of 16 are ahead (4096 x 4096: 32 rows 14 against 17, 64 rows
  // 17 against 18)
  if (rows <= 6 || (d.E == 1 && rows <= 32)) return Kernel::kFewRows;
  // Small grids, by the tiles that an expert of somewhat more rows than the average
  // (their spread is about its root; one alone has as many as there are) needs. Up to a
  // tile of 64 x 64 a CU: those (one expert of 96 rows, 4096 x 4096: 17 us against 20
  // with a ring). Up to two: with a ring of four buffers (8 experts, 4096 x 4096: 16 rows
  // 25 against 29, 48 rows 26 against 30 with rings of 128; one expert of 512 rows 26
  // against 30). Up to one of 128 x 128 a CU: a ring of those (64 rows 30 against 36 to 43,
  // 96 rows 31 against 37; 7 experts of 476 rows, 1040 x 776: 13.2 against 13.9; one expert
  // of 1024 rows 30 against 41; 128 rows, where many have two tiles, 55 against 43
  // without a ring). Past these counts some CUs have a tile more than the others, and
  // most grids lose by it: at two tiles of 64 and a quarter, 36 experts of 30 rows, 2048 x
  // 1024, 27 against 22, 9 of 50 rows, 7168 x 4096, 76 against 72 (4096 x 4096 44 against
  // 47); at one of 128 and an eighth, 9 of 100 rows, 4096 x 4096, 57 against 52, 2048 x
  // 4096, 34 against 30.
  int64_t root = 0;
  while (root * root < rows) ++root;
  const int64_t more = rows + root, most = d.E == 1 ? rows : more;
  const int64_t ct64 = (N + 63) / 64 * d.E, ct128 = (N + 127) / 128 * d.E;
  if ((more + 63) / 64 * ct64 <= num_cus) return Kernel::kTile64;
  if ((most + 63) / 64 * ct64 <= 2 * num_cus) return Kernel::kRing64;
  if ((most + 127) / 128 * ct128 <= num_cus) return Kernel::kRing128;
  // up to 40 rows tiles of 64 x 128, three buffers, weights past the caches: 8 rows 62
  // us against 68 with tiles of 128, 32 rows 74 against 81, 40 rows 77 against 83, 56
  // rows 97 against 88 (64 experts, 7168 x 4096: 39 rows 326 against 341, 47 rows 354
  // against 349)
  if (rows <= 40) return Kernel::kRing64x128;
  // 256 x 256 tiles from 105 rows: 112 rows 102 us against 113, 96 rows 99 against
  // 92; from 41 where the contraction is deep (64 experts, 7168 x 4096: 63 rows 359
  // against 363, 95 rows 374 against 388). They have to fill the CUs, or half of them
  // where their rows would fill two tiles of 128 (8 experts, 4096 x 4096: 256 rows 60
  // against 78, 128 rows 50 against 43).
  const int64_t tiles256 = (rows + 255) / 256 * ((N + 255) / 256) * d.E;
  if ((rows > 104 || d.H >= 4096) && tiles256 >= (rows > 128 ? num_cus / 2 : num_cus)) {
    // the weights past the caches while most experts have one row tile: 160 rows 119
    // us against 127, 192 rows 125 against 132, 224 rows still 151 against 160; 256 rows
    // of 8 experts 66 against 60, 4096 rows of 8 (4096 x 28672) 3645 against 3500
    return rows <= 192 ? Kernel::kTile256Once : Kernel::kTile256;
  }
  // weights past the caches up to 104 rows: 48 rows 87 us against 91, 96 rows 92
  // against 100, but 128 rows 134 against 132
  return rows <= 104 ? Kernel::kTile128Once : Kernel::kTile128;
}

}  // namespace epmi
