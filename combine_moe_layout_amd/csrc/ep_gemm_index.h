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

// Ragged groups.  Group e owns rows [first, first + count) of the row operand
// and matrix e of the other one.  A dense product is one group of R rows.
struct RowGroups {
  const int32_t* first;  // [E + 1] first rows (contiguous layout); NULL: one group of all rows
  const int32_t* count;  // [E] rows wanted by each group (padded layout); NULL when contiguous
  int32_t E;
  int32_t capacity;      // rows per group (padded layout)
  int64_t rows;          // R
  int64_t wanted;        // pairs routed: at most this many rows are used
};

// Row tiles that R rows in E groups can make at most.
inline int64_t max_row_tiles(const RowGroups& g, int32_t height) {
  if (g.first == nullptr) return (g.rows + height - 1) / height;
  const int64_t most = g.wanted / height + (g.wanted < g.E ? g.wanted : g.E);
  if (g.capacity == 0) return most;
  const int64_t padded = (int64_t)g.E * tiles_of(g.capacity, height);
  return padded < most ? padded : most;
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
