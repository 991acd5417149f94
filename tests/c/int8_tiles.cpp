// int8_tiles.cpp -- the tiles of a product of 8-bit integers, as the library chooses them
// (csrc/ep_int8_tiles.h).  Each line of the input: groups, rows in all, columns, swiglu (0 or 1);
// each line of the output: few (0 or 1), height, width.
#include <stdio.h>

#include "ep_int8_tiles.h"

int main() {
  int groups, glu;
  long long rows, columns;
  while (scanf("%d %lld %lld %d", &groups, &rows, &columns, &glu) == 4) {
    const int32_t some = 0;  // (a layout has arrays; the choice does not read them)
    const ep::RowGroups g = {groups > 1 ? &some : nullptr, &some, groups, 0, rows, rows};
    const ep::Int8Tiles t = ep::int8_tiles(g, columns, glu != 0, 256);
    printf("%d %d %d\n", (int)t.few, (int)t.height, (int)t.width);
  }
  return 0;
}
