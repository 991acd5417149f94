"""Products of 8-bit integers in the tiles of 128, 192 and 256 rows by 256 columns, of every number of row
blocks that a wave has in them; what test_int8_tiles.py holds against the library's choice of tiles and
test_gpu_int8_tiles.py runs.  Columns are those of the product: with swiglu half of them are results."""

# rows, channels, columns of the product, height of the tiles, row blocks of 32 rows in them
LINEAR = [(1172, 1040, 4096, 128, {1, 4}), (1200, 896, 4096, 128, {2, 4}), (1232, 1040, 4096, 128, {3, 4}),
          (2300, 1040, 4096, 192, {6}), (2460, 912, 4096, 192, {5, 6}), (3100, 1040, 4096, 256, {7, 8}),
          (3500, 1024, 4096, 256, {6, 8}), (4000, 1168, 4096, 256, {5, 8}), (4060, 272, 4096, 256, {7, 8})]
# tokens, top-k, experts, capacity, channels, columns of the product, height
EXPERTS = [(3000, 2, 4, 0, 1040, 2048, 256), (3000, 2, 4, 1700, 912, 2048, 256), (1024, 2, 8, 0, 1040, 4096, 192),
           (5000, 2, 40, 0, 400, 1600, 128)]


def row_blocks(rows, height):
    """As a group's rows are shared out among its row tiles: evenly, in steps of 16."""
    tiles = -(-rows // height)
    each = min(height, (-(-rows // tiles) + 15) // 16 * 16)
    return {-(-min(each, rows - i * each) // 32) for i in range(tiles)}
