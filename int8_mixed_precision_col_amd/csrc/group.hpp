// Rows in groups: the table of row tiles that the products with a weight per group walk (a
// group: an expert's rows, or an adapter's).
#pragma once

#include "common.hpp"

namespace i8mm {

// entry 0: {tiles}; entry 1 + i: tile i = {group, its first row, its rows (1 .. TM)}. Tiles never
// cross a group's border. Group -1: rows behind the last group's.
constexpr int kMaxGroupsOfRows = 1024;
__host__ __device__ __forceinline__ int64_t group_tiles_most(int64_t rows, int64_t groups, int tm) {
  return rows / tm + (groups + 1 < rows ? groups + 1 : rows);
}

// First row of group g, from ascending offsets [G + 1]; whatever they hold, it is in [0, P].
__device__ __forceinline__ int group_first(const int* offsets, int g, int P) { return min(max(offsets[g], 0), P); }

// Tiles of tm rows before each of the groups 0 .. G (group G: the rows behind the others) and, at G +
// 1, of all: in LDS, by a workgroup of NT threads. Offsets that do not ascend give some numbers.
typedef int GroupTilesBefore[kMaxGroupsOfRows + 2];
template <int NT>
__device__ __forceinline__ void count_group_tiles(const int* offsets, int G, int P, int tm, GroupTilesBefore& first) {
  __shared__ int part[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int per = (G + NT) / NT;  // consecutive groups of a thread, of G + 1
  auto rows_of = [&](int g) { return max((g < G ? group_first(offsets, g + 1, P) : P) - group_first(offsets, g, P), 0); };
  int sum = 0;
  for (int g = tid * per; g < min((tid + 1) * per, G + 1); ++g) sum += (rows_of(g) + tm - 1) / tm;
  int upto = wave_prefix_sum(sum);
  if (lane == 63) part[tid >> 6] = upto;
  __syncthreads();
  for (int w = 0; w < tid >> 6; ++w) upto += part[w];
  int at = upto - sum;
  for (int g = tid * per; g < min((tid + 1) * per, G + 1); ++g) {
    first[g] = at;
    at += (rows_of(g) + tm - 1) / tm;
    if (g == G) first[G + 1] = at;
  }
  __syncthreads();
}

// The group that tile t < first[G + 1] is of.
__device__ __forceinline__ int group_of_tile(const GroupTilesBefore& first, int G, int t) {
  int lo = 0, hi = G;  // the group g with first[g] <= t < first[g + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// {group, first row, rows, 0} of tile number `in` of group g, for tiles of tm rows.
__device__ __forceinline__ int4 group_tile(const int* offsets, int G, int P, int g, int in, int tm) {
  const int row = group_first(offsets, g, P) + in * tm;
  const int end = g < G ? group_first(offsets, g + 1, P) : P;
  return make_int4(g < G ? g : -1, row, min(tm, end - row), 0);
}

// Makes the table of groups 0 .. G - 1 and of the rows behind them, for tiles of tm rows; one
// workgroup of NT threads. Offsets that do not ascend give some table of at most `most` tiles,
// with every row in [0, P).
template <int NT>
__device__ __forceinline__ void make_group_tiles(const int* offsets, int G, int P, int tm, int most, int4* table) {
  __shared__ GroupTilesBefore first;
  count_group_tiles<NT>(offsets, G, P, tm, first);
  const int tiles = min(first[G + 1], most);
  if (threadIdx.x == 0) table[0] = make_int4(tiles, 0, 0, 0);
  for (int t = threadIdx.x; t < tiles; t += NT) {
    const int g = group_of_tile(first, G, t);
    table[1 + t] = group_tile(offsets, G, P, g, t - first[g], tm);
  }
}

// The order in which workgroups take row tiles and feature tiles. Each XCD (workgroup number mod 8)
// takes a contiguous run of the products; the run goes through the groups, all tiles_n feature
// tiles of one after the other, up to 8 row tiles of the group for each, so that workgroups that
// run together share the weight's slabs and the rows' in their XCD's L2.
__device__ __forceinline__ int group_order(int bid, int blocks) {
  const int xcd = bid & 7, extra = blocks & 7;
  return (bid >> 3) + xcd * (blocks >> 3) + min(xcd, extra);
}
// Number `in` of a group's products, of `tiles` row tiles: its row tile and feature tile.
__device__ __forceinline__ void group_product(int in, int tiles, int tiles_n, int& tm, int& tn) {
  const int band = in / (8 * tiles_n), left = in - band * 8 * tiles_n, high = min(tiles - 8 * band, 8);
  tm = 8 * band + left % high;
  tn = left / high;
}

// Part `part` of `parts` of the table of that order: entry 0 {products}, entry 1 + b {group, first
// row, rows, feature tile} of workgroup b. At most tiles_n * most products.
template <int NT>
__device__ __forceinline__ void make_group_order(const int* offsets, int G, int P, int rows, int tiles_n, int most,
                                                 int4* table, int part, int parts) {
  __shared__ GroupTilesBefore first;
  count_group_tiles<NT>(offsets, G, P, rows, first);
  const int blocks = tiles_n * min(first[G + 1], most);
  if (part == 0 && threadIdx.x == 0) table[0] = make_int4(blocks, 0, 0, 0);
  for (int b = part * NT + threadIdx.x; b < blocks; b += parts * NT) {
    const int at = group_order(b, blocks), g = group_of_tile(first, G, at / tiles_n);
    int tm, tn;
    group_product(at - first[g] * tiles_n, first[g + 1] - first[g], tiles_n, tm, tn);
    int4 t = group_tile(offsets, G, P, g, tm, rows);
    t.w = tn;
    table[1 + b] = t;
  }
}

// The same with tiles of different costs: a last tile of at most `half` rows of a group is
// kHalfTileCost / kTileCost of the others. The XCDs' runs are of equal cost rather than number, and
// each takes the groups of the costliest tiles first, so that its last ones are short. A workgroup per
// group, or several groups to one (part of parts); workgroups number up to 8 of the longest
// run, entries past a run's end have no rows. Runs too long for `capacity` entries (a multiple of
// 8), which would take costs far apart, are cut by number.
constexpr int kTileCost = 16, kHalfTileCost = 9;
template <int NT>
__device__ __forceinline__ void make_balanced_order(const int* offsets, int G, int P, int rows, int half, int tiles_n,
                                                    int most, int capacity, int4* table, int part, int parts) {
  __shared__ GroupTilesBefore first, cost;  // before a group: tiles, and their cost
  __shared__ int bound[9];                  // the runs, in products
  __shared__ int part_sums[NT / 64];
  const int tid = threadIdx.x;
  count_group_tiles<NT>(offsets, G, P, rows, first);
  for (int g = tid; g <= G + 1; g += NT) first[g] = min(first[g], most);  // more come only of offsets that do not ascend
  __syncthreads();
  // halves before a group, then the cost
  {
    const int per = (G + NT) / NT;
    auto is_half = [&](int g) {
      const int n = (g < G ? group_first(offsets, g + 1, P) : P) - group_first(offsets, g, P), rest = n % rows;
      return n > 0 && rest > 0 && rest <= half ? 1 : 0;
    };
    int sum = 0;
    for (int g = tid * per; g < min((tid + 1) * per, G + 1); ++g) sum += is_half(g);
    int upto = wave_prefix_sum(sum);
    if ((tid & 63) == 63) part_sums[tid >> 6] = upto;
    __syncthreads();
    for (int w = 0; w < tid >> 6; ++w) upto += part_sums[w];
    int at = upto - sum;
    for (int g = tid * per; g < min((tid + 1) * per, G + 1); ++g) {
      cost[g] = kTileCost * first[g] - (kTileCost - kHalfTileCost) * at;
      at += is_half(g);
      if (g == G) cost[G + 1] = kTileCost * first[G + 1] - (kTileCost - kHalfTileCost) * at;
    }
    __syncthreads();
  }
  const int all = tiles_n * first[G + 1];
  if (tid < 9) {
    const int64_t target = static_cast<int64_t>(cost[G + 1]) * tiles_n * tid / 8;
    int lo = 0, hi = G;  // the last group that starts at or before the target
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(cost[mid]) * tiles_n <= target) lo = mid;
      else hi = mid - 1;
    }
    const int64_t in = target - static_cast<int64_t>(cost[lo]) * tiles_n;
    const int c = cost[lo + 1] - cost[lo], n = first[lo + 1] - first[lo];
    bound[tid] = tid == 8 ? all : min(first[lo] * tiles_n + (c > 0 ? static_cast<int>(in * n / c) : 0), all);
  }
  __syncthreads();
  int longest = 0;
  bool ascending = true;
  for (int x = 0; x < 8; ++x) {
    longest = max(longest, bound[x + 1] - bound[x]);
    ascending = ascending && bound[x + 1] >= bound[x] && bound[x] >= 0;
  }
  __syncthreads();
  if (8 * longest > capacity || !ascending) {
    if (tid < 9) bound[tid] = static_cast<int>(static_cast<int64_t>(all) * tid / 8);
    longest = (all + 7) / 8;
    __syncthreads();
  }
  if (part == 0) {
    if (tid == 0) table[0] = make_int4(8 * longest, 0, 0, 0);
    for (int e = tid; e < 8 * longest; e += NT)
      if (e / 8 >= bound[(e & 7) + 1] - bound[e & 7]) table[1 + e] = make_int4(0, 0, 0, 0);
  }
  // a group's products in run x, [from, to)
  auto from = [&](int g, int x) { return max(first[g] * tiles_n, bound[x]); };
  auto to = [&](int g, int x) { return min(first[g + 1] * tiles_n, bound[x + 1]); };
  for (int g = part; g <= G; g += parts) {
    const int tiles = first[g + 1] - first[g], c = cost[g + 1] - cost[g];
    for (int x = 0; x < 8; ++x) {
      const int p0 = from(g, x), p1 = to(g, x);
      if (p0 >= p1) continue;
      // the products of the run's groups that come first
      int before = 0;
      for (int h = tid; h <= G; h += NT) {
        const int n = to(h, x) - from(h, x);
        if (n <= 0) continue;
        const int64_t mine = static_cast<int64_t>(c) * (first[h + 1] - first[h]);
        const int64_t its = static_cast<int64_t>(cost[h + 1] - cost[h]) * tiles;
        if (its > mine || (its == mine && h < g)) before += n;
      }
      const int sum = __builtin_amdgcn_readlane(wave_prefix_sum(before), 63);
      __syncthreads();
      if ((tid & 63) == 0) part_sums[tid >> 6] = sum;
      __syncthreads();
      before = 0;
      for (int w = 0; w < NT / 64; ++w) before += part_sums[w];
      for (int p = p0 + tid; p < p1; p += NT) {
        int tm, tn;
        group_product(p - first[g] * tiles_n, tiles, tiles_n, tm, tn);
        int4 t = group_tile(offsets, G, P, g, tm, rows);
        t.w = tn;
        table[1 + 8 * (before + p - p0) + x] = t;
      }
    }
  }
}

}  // namespace i8mm
