// What the products with a weight per group of rows share (mx4_grouped.hip, int8_grouped.hip).
//
// A workgroup takes a row tile and TN features of its group's weight.
// The rows of a tile are any rows of X: each lane of the DMA that fills the ring brings 16 bytes
// of the row that its place holds, so the rows are gathered on their way into LDS and the K loop
// is the ungrouped product's. gated: a tile's 16-row groups of the weight are gate and up in
// turn, so that a lane holds both of a feature and the epilogue writes silu(gate) up.
#pragma once

#include "gemm_kernel.hpp"
#include "group.hpp"
#include "group_launch.hpp"

namespace i8mm {

// 256 x 256 and 128 x 128 (features x rows) on 8 waves, 128 x 64 on 4; 4-stage rings.
using GroupL = GemmCfg<256, 256, 64, 2, 4, 4>;
using GroupS = GemmCfg<128, 128, 64, 2, 4, 4>;
using GroupT = GemmCfg<128, 64, 64, 2, 2, 4>;
// What MX4 takes a tile of at most 128 rows by where others have 256, on their ring: all waves on these
// rows, and a quarter less to bring per slab (768 tokens, 8 of 64 experts of 4096 x 1280 109 -> 105
// us). With int8 both in one kernel spill.
using GroupH = GemmCfg<256, 128, 64, 2, 4, 4>;
template <>
__device__ __forceinline__ char* stage_buf<GroupH, 0>() { return stage_buf<GroupL, 0>(); }
template <>
__device__ __forceinline__ char* stage_buf<GroupH, 1>() { return stage_buf<GroupL, 1>(); }
template <>
__device__ __forceinline__ char* stage_buf<GroupH, 2>() { return stage_buf<GroupL, 2>(); }
template <>
__device__ __forceinline__ char* stage_buf<GroupH, 3>() { return stage_buf<GroupL, 3>(); }

// A tile's group (-1: rows behind the last group's), its first row and its rows, 1 .. TM.
struct RowTile {
  int group, first, rows;
};

// 16-row group of the group's weight behind place v of a tile whose first output feature is n0.
// Past the last feature it is the last one's (those outputs are not stored).
template <bool GATED>
__device__ __forceinline__ int weight_group(int v, int n0, int N) {
  if constexpr (GATED) return (v & 1) * (N / 32) + min(n0 / 16 + (v >> 1), N / 32 - 1);
  return min(n0 / 16 + v, N / 16 - 1);
}

// Row of X behind row r of a tile; M, a row of zeros, where there is none.
__device__ __forceinline__ int source_row(const GroupShape& g, const RowTile& tile, int r) {
  if (r >= tile.rows) return g.M;
  const int p = tile.first + r;
  const int s = g.rows ? g.rows[p] : p;
  return s >= 0 && s < g.M ? s : g.M;
}

template <class C, bool GATED>
__device__ __forceinline__ void zero_tile(const GroupShape& g, const RowTile& tile, int n0) {
  constexpr int OUT = GATED ? C::TN / 2 : C::TN;
  const int N = GATED ? g.N / 2 : g.N;
  for (int t = threadIdx.x; t < tile.rows * (OUT / 8); t += C::NT) {
    const int n = n0 + t % (OUT / 8) * 8;
    if (n < N) *reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.Y) + static_cast<size_t>(tile.first + t / (OUT / 8)) * N + n) = v4u{};
  }
}

// The row tile and feature tile of this workgroup (false: there is none for it), in the order of
// group_order. With a table of it (g.table) that is one load; otherwise every wave works it out for
// itself from the offsets, 64 groups at a time, which takes 2.4 us of a tile's start. Offsets that do
// not ascend give some tiles, at most g.tiles_most, with all rows in [0, P).
template <class C, bool TABLE>
__device__ __forceinline__ bool group_tile_of(const GroupShape& g, int tiles_n, RowTile& tile, int& tn) {
  if constexpr (TABLE) {
    const int4 head = g.table[0], t = g.table[1 + blockIdx.x];  // on their way together
    if (static_cast<int>(blockIdx.x) >= head.x || t.z <= 0) return false;
    tile.group = t.x;
    tile.first = t.y;
    tile.rows = t.z;
    tn = t.w;
    return true;
  }
  const int lane = threadIdx.x & 63, chunks = g.G / 64 + 1;  // of the G + 1 groups
  auto rows_of = [&](int e, int& first) {
    first = e <= g.G ? group_first(g.offsets, e, g.P) : g.P;
    return max((e < g.G ? group_first(g.offsets, e + 1, g.P) : g.P) - first, 0);
  };
  int sums = 0, first = 0, rows = 0, upto = 0;  // lane c: the tiles of chunk c
  for (int c = 0; c < chunks; ++c) {
    rows = rows_of(64 * c + lane, first);
    upto = wave_prefix_sum((rows + C::TM - 1) / C::TM);
    const int sum = __builtin_amdgcn_readlane(upto, 63);
    if (lane == c) sums = sum;
  }
  const int chunk_upto = wave_prefix_sum(sums);
  const int tiles_m = min(__builtin_amdgcn_readlane(chunk_upto, 63), g.tiles_most), blocks = tiles_n * tiles_m;
  if (static_cast<int>(blockIdx.x) >= blocks) return false;
  int at = group_order(blockIdx.x, blocks);
  const int chunk = __builtin_ctzll(__ballot(chunk_upto > at / tiles_n));
  at -= __builtin_amdgcn_readlane(chunk_upto - sums, chunk) * tiles_n;
  if (chunks > 1) {
    rows = rows_of(64 * chunk + lane, first);
    upto = wave_prefix_sum((rows + C::TM - 1) / C::TM);
  }
  const int e = __builtin_ctzll(__ballot(upto > at / tiles_n)), n = __builtin_amdgcn_readlane(rows, e);
  const int tiles = (n + C::TM - 1) / C::TM;
  int tm;
  group_product(at - (__builtin_amdgcn_readlane(upto, e) - tiles) * tiles_n, tiles, tiles_n, tm, tn);
  tile.group = 64 * chunk + e < g.G ? 64 * chunk + e : -1;
  tile.first = __builtin_amdgcn_readlane(first, e) + tm * C::TM;
  tile.rows = min(n - tm * C::TM, C::TM);
  return true;
}

// silu(g) u = g u / (1 + exp(-g)), within 1.23 |g| + 7 units of 2^-24 relative: exp as 2^p, p the rounded
// product of -g and log2(e) in fp32 (1 unit of p and 0.23 of the constant, |g| times each in exp), by the
// exponential and reciprocal instructions (each within one unit in the last place, so 2), a sum and two
// products. The output keeps 8 or 11 bits: at |g| = 60 this is 2^-17.6. Where exp is above 2^126 the result
// is 0 (it is below 2^-119 u). 64 of them per lane follow a 256 x 256 tile: with expf and an IEEE quotient
// they took 7 of its 44 us at K = 4096, so 3. (What p's rounding left, q - p ln(2), brought back in by three
// products and a clamp: 8 units for any g, and 2% of the whole: 4096 tokens, 8 of 64 experts of 4096 x 1280,
// MX4, 236.5 -> 241.4 us.)
__device__ __forceinline__ float silu_up(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

// Rounds the wave's part of the tile into its slice of the ring and stores whole row segments, 16
// bytes per lane. 16 x 16 accumulator layout: lane l, register e holds row m = l % 16, feature
// 4 (l / 16) + e; value(i, j, e) is that of block (i, j).
template <class C, class T, bool GATED, class F>
__device__ __forceinline__ void store_tile(const GroupShape& g, const RowTile& tile, int n0, int wn, int wm, int lane,
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
    if (m < tile.rows && n < N)
      *reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.Y) + static_cast<size_t>(tile.first + m) * N + n) = v;
  }
}

}  // namespace i8mm
