// gemm_index.cpp -- walks the index arithmetic of the matrix-product kernels
// (csrc/ep_gemm_index.h) on the host: every row of the matrix operand that a tile
// loads lies inside its expert's matrix (results do not show a row past it: its
// products are dropped), and counts up to 2^31 - 1 rows and the grids made of them
// come out whole.  Exit status 0 if all hold; the first that does not is printed.
#include <stdio.h>

#include <initializer_list>

#include "ep_gemm_index.h"

namespace {

int fail(const char* what, bool glu, int wave_cols, int out_cols, int col, int p, int row) {
  printf("%s: %s, %d columns a wave, %d columns, column tile %d, place %d: row %d\n", what,
         glu ? "swiglu" : "plain", wave_cols, out_cols, col, p, row);
  return 1;
}

// The matrix rows of one tile shape: 4 waves side by side of `wave_cols` places.
// `rows`: neighbouring rows that a wave counts from its first (FP8), or 1.
int walk(bool glu, int wave_cols, int out_cols, int rows) {
  const int places = 4 * wave_cols, tile_cols = glu ? places / 2 : places;
  const int width = glu ? 2 * out_cols : out_cols;
  for (int col = 0; col * tile_cols < out_cols; ++col)
    for (int p = 0; p < places; p += rows) {
      const int first = ep::matrix_row(glu, p, wave_cols, col * tile_cols, out_cols, rows);
      if (first < 0 || first + rows > width) return fail("outside", glu, wave_cols, out_cols, col, p, first);
      // where the column exists, the row is its own
      const int in = p % wave_cols, half = wave_cols / 2;
      const int n = glu ? col * tile_cols + p / wave_cols * half + in % half : col * tile_cols + p;
      if (n < out_cols && first != n + (glu && in >= half ? out_cols : 0))
        return fail("wrong row", glu, wave_cols, out_cols, col, p, first);
    }
  return 0;
}

// Tiles and chunks of a count, up to the largest.
int count_tiles() {
  const int64_t last = INT32_MAX;
  for (int height : {16, 32, 64, 128, 192, 256})
    for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)height - 1, (int64_t)height, (int64_t)height + 1,
                      last - height, last - height + 1, last - height + 2, last - 1, last})
      if (ep::tiles_of((int32_t)n, height) != (n + height - 1) / height) {
        printf("%d tiles of %d in %lld rows\n", ep::tiles_of((int32_t)n, height), height, (long long)n);
        return 1;
      }
  return 0;
}

// The grid's bound on row tiles: E groups of `capacity` rows, `wanted` pairs among them.
int bound_tiles() {
  const int32_t last = INT32_MAX;
  for (int32_t E : {1, 2, 3})
    for (int32_t capacity : {1, 64, last / 4, last - 300, last - 15, last}) {
      if ((int64_t)E * capacity > last) continue;
      for (int64_t wanted : {(int64_t)1, (int64_t)1000, (int64_t)last})
        for (int height : {16, 64, 128, 192, 256}) {
          const ep::RowGroups g = {&capacity, &capacity, E, capacity, (int64_t)E * capacity, wanted};
          const int64_t each = ((int64_t)capacity + height - 1) / height, got = ep::max_row_tiles(g, height);
          const int64_t rows = wanted < g.rows ? wanted : g.rows;
          if (got < (rows + height - 1) / height || got > E * each) {
            printf("%lld tiles of %d for %d x %d rows, %lld pairs\n", (long long)got, height, E, capacity,
                   (long long)wanted);
            return 1;
          }
        }
    }
  return 0;
}

}  // namespace

int main() {
  if (count_tiles() || bound_tiles()) return 1;
  for (int glu = 0; glu < 2; ++glu)
    for (int wave_cols = 32; wave_cols <= 64; wave_cols *= 2) {
      // FP8: a wave of 8 brings half a column of waves' places, counted from the first
      for (int n = 128; n <= 8192; n += 128)
        if (walk(glu, wave_cols, n, wave_cols / 2) || walk(glu, wave_cols, n, 1)) return 1;
      // 16-bit: any multiple of 8 columns, row by row
      for (int n = 8; n <= 1200; n += 8)
        if (walk(glu, wave_cols, n, 1)) return 1;
    }
  return 0;
}
