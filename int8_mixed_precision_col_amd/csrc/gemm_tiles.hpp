// Choice of a GEMM tile shape by estimated time (shared by the int8 and MX4 launchers).
#pragma once

#include <hip/hip_runtime.h>

namespace i8mm {

// Which tile shape: the one with the least estimated time, counted in waves of tiles
// over the CUs times the tile's cost relative to a 256 x 256 tile (its area over its
// measured rate: 1, 0.9 and 0.85 of the 256 x 256 rate on full waves). A last, partial
// wave of tiles costs at least 0.6 of a full one: its tiles run alone but not faster
// in proportion. On MI355X this picks the measured fastest shape, or one within 3% of
// it, for 2048 x 4096 x {4096, 12288, 16384}, 4096 x 4096 x 4096, 4096 x 20480 x 5120,
// 4096 x 12288 x 49152, 1024 x 4096 x 4096 and 512 x 8192 x 8192.
enum class Tile { L, M, S };
inline int device_cus() {
  static int cus = 0;
  if (cus == 0) {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && v > 0)
      cus = v;
    else
      return 256;
  }
  return cus;
}
inline double wave_cost(long tiles) {
  const double w = static_cast<double>(tiles) / device_cus();
  const double full = static_cast<double>(static_cast<long>(w)), frac = w - full;
  return full + (frac > 0.0 ? (frac > 0.6 ? frac : 0.6) : 0.0);
}
// tiles(tn, tm): tile count for a tile of tn features x tm tokens
template <class F>
inline Tile pick_tile(F tiles) {
  const double cl = wave_cost(tiles(256, 256));
  const double cm = wave_cost(tiles(128, 256)) * (0.5 / 0.9);
  const double cs = wave_cost(tiles(128, 128)) * (0.25 / 0.85);
  if (cl <= cm && cl <= cs) return Tile::L;
  return cm <= cs ? Tile::M : Tile::S;
}

// Cost, in waves of 256 x 256 tiles, of the best single tile shape for the tile counts
// tiles(tn, tm).
template <class F>
inline double best_cost(F tiles, Tile* t) {
  *t = pick_tile(tiles);
  if (*t == Tile::L) return wave_cost(tiles(256, 256));
  if (*t == Tile::M) return wave_cost(tiles(128, 256)) * (0.5 / 0.9);
  return wave_cost(tiles(128, 128)) * (0.25 / 0.85);
}

}  // namespace i8mm
