// The choice of a tile shape for the products grouped by expert.
#include "group.hpp"
#include "group_launch.hpp"

namespace i8mm {

int group_tile_rows(GroupTile t) { return t == GroupTile::S ? 128 : t == GroupTile::T ? 64 : 256; }
int group_tile_features(GroupTile t) { return t == GroupTile::L ? 256 : 128; }

// By the mean rows of a group: few rows are bound by the weights' bytes, which smaller tiles (more
// of them at once) bring in faster, and pad less; many rows by the slabs that come into LDS per
// product, fewest in the largest tiles. Measured (us per call in a graph, X's quantization
// included, 128 x 64 / 128 x 128 / 256 x 256), MX4: mean 3 rows of 64 groups, K x N 2048 x 1536 22.4
// / 25.0 / 37.4; 32 rows, 4096 x 2560 85 / 91 / 108; 128 rows 134 / 132 / 133, of 2048 x 1536 55 / 58 /
// 60; 512 rows, 4096 x 2560 369 / 343 / 305, of 8 groups, 4096 x 8192 157 / 142 / 131. int8: 23 rows of
// 10 groups, 1040 x 528 22.6 / 23.0 / 33; 64 rows of 64, 2048 x 1536 78 / 75 / 99; 256 rows of 16 54 / 45 /
// 57; 512 rows of 64 237 / 214 / 195.
GroupTile pick_group_tile(int64_t P, int64_t groups, bool int8) {
  const int64_t rows = P / (groups < P ? groups : P);
  if (rows <= (int8 ? 48 : 128)) return GroupTile::T;
  return rows <= 256 ? GroupTile::S : GroupTile::L;
}

}  // namespace i8mm
