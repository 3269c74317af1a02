// The table of row tiles (group.hpp) in a launch of its own, and the choice of a tile shape.
#include "group.hpp"
#include "group_launch.hpp"

namespace i8mm {

__global__ __launch_bounds__(256) void k_group_tiles(const int32_t* offsets, int G, int P, int tm, int most, int4* table) {
  make_group_tiles<256>(offsets, G, P, tm, most, table);
}

hipError_t launch_group_tiles(const int32_t* offsets, int G, int P, int tm, int4* table, hipStream_t s) {
  hipLaunchKernelGGL(k_group_tiles, dim3(1), dim3(256), 0, s, offsets, G, P, tm,
                     static_cast<int>(group_tiles_most(P, G, tm)), table);
  return hipGetLastError();
}

int group_tile_rows(GroupTile t) { return t == GroupTile::S ? 128 : t == GroupTile::T ? 64 : 256; }

GroupTile pick_group_tile(int64_t P, int64_t groups, int64_t N) {
  const int64_t per = P / (groups < P ? groups : P);
  if (per <= 96) return GroupTile::T;
  if (per <= 256) return GroupTile::S;
  return GroupTile::L;
}

}  // namespace i8mm
