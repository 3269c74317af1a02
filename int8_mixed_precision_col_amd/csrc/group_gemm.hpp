// What the products with a weight per group of rows share (mx4_grouped.hip, int8_grouped.hip).
//
// A workgroup takes a row tile of the table (group.hpp) and TN features of that group's weight.
// The rows of a tile are any rows of X: each lane of the DMA that fills the ring brings 16 bytes
// of the row that its place holds, so the rows are gathered on their way into LDS and the K loop
// is the ungrouped product's. gated: a tile's 16-row groups of the weight are gate and up in
// turn, so that a lane holds both of a feature and the epilogue writes silu(gate) up.
#pragma once

#include "gemm_kernel.hpp"
#include "group.hpp"
#include "group_launch.hpp"

namespace i8mm {

// 16-row group of the group's weight behind place v of a tile whose first output feature is n0.
// Past the last feature it is the last one's (those outputs are not stored).
template <bool GATED>
__device__ __forceinline__ int weight_group(int v, int n0, int N) {
  if constexpr (GATED) return (v & 1) * (N / 32) + min(n0 / 16 + (v >> 1), N / 32 - 1);
  return min(n0 / 16 + v, N / 16 - 1);
}

// Row of X behind row r of a tile; M, a row of zeros, where there is none.
__device__ __forceinline__ int source_row(const GroupShape& g, const int4& tile, int r) {
  if (r >= tile.z) return g.M;
  const int p = tile.y + r;
  const int s = g.rows ? g.rows[p] : p;
  return s >= 0 && s < g.M ? s : g.M;
}

template <class C, bool GATED>
__device__ __forceinline__ void zero_tile(const GroupShape& g, const int4& tile, int n0) {
  constexpr int OUT = GATED ? C::TN / 2 : C::TN;
  const int N = GATED ? g.N / 2 : g.N;
  for (int t = threadIdx.x; t < tile.z * (OUT / 8); t += C::NT) {
    const int n = n0 + t % (OUT / 8) * 8;
    if (n < N) *reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.Y) + static_cast<size_t>(tile.y + t / (OUT / 8)) * N + n) = v4u{};
  }
}

// The tile of workgroup b (false: none); table and order as in tile_of, over the tiles that
// there are.
__device__ __forceinline__ bool group_tile_of(const GroupShape& g, int tiles_n, int4& tile, int& tn) {
  const int tiles_m = g.table[0].x, blocks = tiles_n * tiles_m;
  if (static_cast<int>(blockIdx.x) >= blocks) return false;
  int tm;
  tile_of(blockIdx.x, blocks, tiles_m, min(tiles_m, 8), tn, tm);
  tile = g.table[1 + tm];
  return true;
}

__device__ __forceinline__ float silu_up(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// Rounds the wave's part of the tile into its slice of the ring and stores whole row segments, 16
// bytes per lane. 16 x 16 accumulator layout: lane l, register e holds row m = l % 16, feature
// 4 (l / 16) + e; value(i, j, e) is that of block (i, j).
template <class C, class T, bool GATED, class F>
__device__ __forceinline__ void store_tile(const GroupShape& g, const int4& tile, int n0, int wn, int wm, int lane,
                                           F value) {
  typedef typename T::elem v4t __attribute__((ext_vector_type(4)));
  constexpr int WF = GATED ? C::WTN / 2 : C::WTN;  // output features of a wave
  constexpr int CH = WF / 8, RB = WF * 2, RPI = 64 / CH;
  const int l16 = lane & 15, lq = lane >> 4, N = GATED ? g.N / 2 : g.N;
  // 16 rows of a store go to 16 different banks' places: 256-byte rows by all of the row, 128 by
  // half, 64 by a quarter
  auto swizzle = [](int r) { return CH == 16 ? r & 15 : CH == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
  char* ys = wave_slice<C>(wn + C::WGN * wm);
#pragma unroll
  for (int i = 0; i < WF / 16; ++i)
#pragma unroll
    for (int j = 0; j < C::BM; ++j) {
      const int r = j * 16 + l16;
      v4t out;
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = T::round(value(i, j, e));
      *reinterpret_cast<v4t*>(ys + r * RB + 16 * ((2 * i + (lane >> 5)) ^ swizzle(r)) + 8 * (lq & 1)) = out;
    }
  const int c = lane % CH;
  const int n = n0 + wn * WF + 8 * c;
#pragma unroll
  for (int t = 0; t < C::WTM / RPI; ++t) {
    const int r = t * RPI + lane / CH;
    const v4u v = *reinterpret_cast<const v4u*>(ys + r * RB + 16 * (c ^ swizzle(r)));
    const int m = wm * C::WTM + r;
    if (m < tile.z && n < N)
      *reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.Y) + static_cast<size_t>(tile.y + m) * N + n) = v;
  }
}

// 256 x 256, 128 x 256, 128 x 128 (features x rows) on 8 waves, 128 x 64 on 4; 4-stage rings.
using GroupL = GemmCfg<256, 256, 64, 2, 4, 4>;
using GroupM = GemmCfg<128, 256, 64, 2, 4, 4>;
using GroupS = GemmCfg<128, 128, 64, 2, 4, 4>;
using GroupT = GemmCfg<128, 64, 64, 2, 2, 4>;

}  // namespace i8mm
