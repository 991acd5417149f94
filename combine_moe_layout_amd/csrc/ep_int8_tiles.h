// ep_int8_tiles.h -- which tiles a product of 8-bit integers is made in: host code without a GPU
// (tests/c/int8_tiles.cpp walks it).
#pragma once

#include <math.h>
#include <stdint.h>

#include "ep_gemm_index.h"

namespace ep {

// Estimated time of a product in tiles of `height` rows, in units of the 6.5 us that one row block
// to a wave takes with 7168 channels.  A big tile of RB row blocks takes RB + 2 (39 us for 128 rows,
// 52 for 192, 65 for 256), and a CU holds one; a small one takes 3.2 by itself and 6.5 where two
// share a CU.  Few tiles run in rounds, the last of which may leave CUs idle; many even out.
// Groups' rows scatter about their mean by its root, so that a mean just below the height makes
// two tiles of every other group.
// Measured, us, 128 / 192 / 256 rows: 7168 x 4096 channels and columns, 1024 rows 40 / 52 / 65, 3000
// rows 87 / 68 / 72, 4096 rows 104 / 130 / 86; 8 experts of 256 rows, 2048 x 4096, 39 / 25 / 30.
inline double int8_estimate(int64_t groups, int64_t rows, int64_t columns, int32_t height,
                            int cus) {
  const int64_t column_tiles = (columns + (height > 64 ? 255 : 127)) / (height > 64 ? 256 : 128);
  const double spread = groups > 1 ? sqrt((double)rows) : 0.0;
  double count = 0, work = 0, longest = 0;
  for (int k = -1; k <= 1; ++k) {
    const int64_t here = (int64_t)((double)rows + k * spread);
    const int64_t n = (here + height - 1) / height;
    if (n <= 0) continue;
    const int64_t each = (here + n - 1) / n, blocks = (each + 31) / 32;
    const double cost = height > 64 ? (double)(blocks + 2) : 3.25;
    count += (double)n / 3;
    work += (double)n * cost / 3;
    longest = cost > longest ? cost : longest;
  }
  const double tiles = (double)(groups * column_tiles) * count;
  if (height == 64) return 3.2 + (tiles > cus ? 3.3 * (tiles - cus) / cus : 0.0);
  if (tiles > 3 * cus) return (double)(groups * column_tiles) * work / cus;
  return ceil(tiles / cus) * longest;
}

struct Int8Tiles {
  bool few;  // the kernel whose waves share out the reduction
  int32_t height, width;
};
// Products whose tiles of 16, 32 or 64 rows and columns all have a CU of their own go to the kernel whose
// waves share out the reduction, in the smallest such tiles: what a CU reads is what takes its time.
// Matrices from HBM, 7168 channels, us: 16 rows, 8192 columns in 16 x 32 12.6, 64 x 32 14.8, 64 x 64
// 21.3; 32 rows in 32 x 32 14.3, 64 x 64 22.1; 100 rows, 4096 columns in 64 x 32 15.4, 64 x 64 22.5.
// 64 x 128 tiles of the other kernel instead: 1 row, 4096 columns 20 (7.7 in 16 x 16), 256 rows 30 (23
// in 64 x 64).  Experts of at most 32 rows are bound by reading their matrices, which those tiles do
// faster where there are many (256 experts of 512 x 2048, 32 rows each: 49 us against 55).
inline Int8Tiles int8_tiles(const RowGroups& r, int64_t out_cols, bool glu, int cus) {
  const int64_t groups = r.wanted > r.E ? r.E : r.wanted, rows = (r.wanted + r.E - 1) / r.E;
  const int64_t columns = out_cols * (glu ? 2 : 1);
  const auto tiles = [&](int64_t height, int64_t width) {
    return groups * ((rows + height - 1) / height) * ((columns + width - 1) / width);
  };
  const int32_t low = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  for (int32_t width = 16; width <= 64; width *= 2)
    if (tiles(low, width) <= cus) return {true, low, width};
  // Where 64 x 128 tiles would share CUs and 128 x 128 tiles do not, those.  Matrices from HBM, 4096
  // columns, us: 7168 channels, 640 rows 38 (else 44), 1024 rows 40 (55); 4096 channels 24 (27), 26 (35);
  // 8 experts of 128 rows, 2048 x 4096, 21 (22).  Where neither share, 512 rows of the first 38 (31).
  if (rows > 32 && tiles(64, 128) > cus && tiles(128, 128) <= cus) return {false, 128, 128};
  int32_t height = 64;
  if (rows > 32)
    for (int32_t h = 128; h <= 256; h += 64)
      if (int8_estimate(groups, rows, columns, h, cus) <= int8_estimate(groups, rows, columns, height, cus)) height = h;
  return {false, height, height == 64 ? 128 : 256};
}

}  // namespace ep
