// The choice of a tile shape for the products grouped by expert.
#include "group.hpp"
#include "group_launch.hpp"

namespace i8mm {

int group_tile_rows(GroupTile t) { return t == GroupTile::S ? 128 : t == GroupTile::T ? 64 : 256; }
int group_tile_features(GroupTile t) { return t == GroupTile::L ? 256 : 128; }

// By the mean rows of a group: few rows are bound by the weights' bytes, which smaller tiles (more
// of them at once) bring in faster, and pad less; many rows by the slabs that come into LDS per
// product, fewest in the largest tiles. Measured, us per call in a graph, X's quantization included,
// with tiles of 64 / 128 / 256 rows.
// MX4, 64 experts, K x N 4096 x 2560, mean rows 48 86 / 91 / 94, 64 95 / 97 / 98, 96 112 / 108 / 105, 128
// 130 / 126 / 114, 256 203 / 183 / 153; of 2048 x 1536, 64 37 / 38 / 41, 128 50 / 50 / 49; of 1280 x 4096, 64
// 67 / 68 / 69, 128 100 / 93 / 85; 8 experts of 4096 x 8192, 32 41 / 41 / 37, 128 61 / 59 / 66, 256 90 / 85 /
// 76. A short K leaves a large tile mostly its start and end: 768 x 2048, 128 31 / 32 / 36, 256 69 / 63 / 58.
// (128 rows are best nowhere by more than 12%, and left out. The rule takes the slower of 64 and 256 at two
// of these points: 8 experts of 4096 x 8192, 32 rows, 41 where 256 take 37, and 128 rows, 66 where 64 take 61.)
// int8, 64 experts of 2048 x 1536, 16 55 / 63 / 83, 32 64 / 66 / 82, 64 73 / 69 / 84, 128 91 / 90 / 89, 256 132 /
// 120 / 128, 512 237 / 214 / 195; 8 experts of 4096 x 4096, 128 69 / 68 / 71, 256 94 / 87 / 78 (where the rule takes
// 128 rows: it does not look at K for int8).
// With few tiles in all, CUs stay idle for the whole time of a large one: 64 / 256 rows, MX4, 27 tiles
// of 256 rows (10 experts of 1040 x 528) 8.8 / 16.3, 128 (16 of 2048 x 2048) 19 / 23, 160 (4 of 4096 x 4096) 44 /
// 37, 192 (16 of 2048 x 2048) 27 / 26; int8, 64 / 128 rows, 256 tiles of 128 (16 of 2048 x 2048) 32 / 35, 384 40 / 39.
GroupTile pick_group_tile(int64_t P, int64_t groups, int64_t N, int64_t K, bool int8) {
  const int64_t used = groups < P ? groups : P, rows = P / used;
  // tiles of f features x r rows, half of one more per group
  auto tiles = [&](int f, int r) { return (N + f - 1) / f * (P / r + used / 2); };
  if (rows > (int8 ? 256 : K <= 1024 ? 160 : 72) && tiles(256, 256) >= 160) return GroupTile::L;
  if (int8 && rows > 48 && tiles(128, 128) >= 320) return GroupTile::S;
  return GroupTile::T;
}

}  // namespace i8mm
