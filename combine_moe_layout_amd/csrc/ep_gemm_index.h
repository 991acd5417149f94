// ep_gemm_index.h -- index arithmetic of the matrix-product kernels that needs
// no GPU: constexpr functions, which device code calls as they are and a host
// compiler takes too (tests/c/gemm_index.cpp walks every operand row that a tile
// loads).
#pragma once

#include <stdint.h>

namespace ep {

// ceil(count / height): row tiles of a group, chunks of a reduction.  A count may be
// as large as 2^31 - 1.
constexpr int32_t tiles_of(int32_t count, int32_t height) {
  return (int32_t)(((uint32_t)count + (uint32_t)height - 1) / (uint32_t)height);
}

// A tile's LDS holds rows of the matrix operand, `wave_cols` to a column of waves.
// Row of the matrix at place p of them, or the first of `rows` neighbouring ones
// from place p on; first_col: the tile's first result column, out_cols: all result
// columns.  For swiglu the first half of a wave's rows are gates, the second half
// the ups of the same columns.  What stands at places past the last column is
// loaded as well (and its products are dropped), so it has to lie inside the
// matrix: there it is the last `rows` rows.  (rows > 1 takes columns in whole
// multiples of rows: of `rows` places either all have a column or none.)
constexpr int32_t matrix_row(bool glu, int32_t p, int32_t wave_cols, int32_t first_col,
                             int32_t out_cols, int32_t rows = 1) {
  int32_t n = first_col + p, ups = 0;
  if (glu) {
    const int32_t half = wave_cols / 2, in = p % wave_cols;
    n = first_col + p / wave_cols * half + in % half;
    ups = in >= half ? out_cols : 0;
  }
  return (n < out_cols - rows ? n : out_cols - rows) + ups;
}

}  // namespace ep
