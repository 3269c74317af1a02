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
// each takes the groups of the costliest tiles first, so that its last ones are short. Workgroups
// number up to 8 of the longest run, entries past a run's end have no rows. Runs too long for
// `capacity` entries (a multiple of 8), which would take costs far apart, are cut by number.
// 32768 pairs, 64 experts of 4096 x 1280: the gate and up product 240.6 -> 234.1 us; costs of 7, 8,
// 11 and 13 in place of 9 come out at 240, 236, 237 and 234.
constexpr int kTileCost = 16, kHalfTileCost = 9;
template <int NT>
__device__ __forceinline__ void make_balanced_order(const int* offsets, int G, int P, int rows, int half, int tiles_n,
                                                    int most, int capacity, int4* table, int part, int parts) {
  __shared__ GroupTilesBefore start, first, cost;  // of a group: its first row; tiles and their cost before it
  __shared__ int bound[9];                         // the runs, in products
  __shared__ int2 sums[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = (G + NT) / NT, g0 = tid * per, g1 = min(g0 + per, G + 1);  // consecutive groups of a thread
  for (int g = g0; g < g1; ++g) start[g] = group_first(offsets, g, P);
  if (tid == 0) start[G + 1] = P;
  if (tid < 9) bound[tid] = 0;
  __syncthreads();
  auto tiles_of = [&](int g) { return (max(start[g + 1] - start[g], 0) + rows - 1) / rows; };
  auto halves_of = [&](int g) {
    const int n = max(start[g + 1] - start[g], 0), rest = n % rows;
    return rest > 0 && rest <= half ? 1 : 0;
  };
  int tiles = 0, halves = 0;
  for (int g = g0; g < g1; ++g) tiles += tiles_of(g), halves += halves_of(g);
  int2 upto = make_int2(wave_prefix_sum(tiles), wave_prefix_sum(halves));
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int2 total = make_int2(0, 0);
  for (int w = 0; w < NT / 64; ++w) {
    if (w == wave) upto.x += total.x, upto.y += total.y;
    total.x += sums[w].x, total.y += sums[w].y;
  }
  const bool ascending = total.x <= most;  // more come only of offsets that do not ascend
  const int all_tiles = min(total.x, most), all = tiles_n * all_tiles;
  const int64_t all_cost = static_cast<int64_t>(kTileCost * all_tiles - (kTileCost - kHalfTileCost) * total.y) * tiles_n;
  {
    int at = upto.x - tiles, at_half = upto.y - halves;
    for (int g = g0; g < g1; ++g) {
      const int n = tiles_of(g), c = kTileCost * n - (kTileCost - kHalfTileCost) * halves_of(g);
      first[g] = min(at, most);
      cost[g] = kTileCost * at - (kTileCost - kHalfTileCost) * at_half;
      if (g == G) first[G + 1] = min(at + n, most), cost[G + 1] = cost[g] + c;
      // the runs that begin in this group; their ends may be a product off by the float's rounding
      const int64_t from = static_cast<int64_t>(cost[g]) * tiles_n, to = from + static_cast<int64_t>(c) * tiles_n;
      if (ascending && n > 0)
        for (int x = 1; x < 8; ++x) {
          const int64_t target = all_cost * x >> 3;
          if (from <= target && target < to)
            bound[x] = tiles_n * at + min(static_cast<int>(static_cast<float>(target - from) * n / c), tiles_n * n);
        }
      at += n;
      at_half += halves_of(g);
    }
    if (tid == 0) bound[8] = all;
  }
  __syncthreads();
  int longest = 0;
  for (int x = 0; x < 8; ++x) longest = max(longest, bound[x + 1] - bound[x]);
  const bool equal = !ascending || 8 * longest > capacity;
  if (equal) longest = (all + 7) / 8;
  auto run = [&](int x) { return equal ? static_cast<int>(static_cast<int64_t>(all) * x >> 3) : bound[x]; };
  if (part == parts - 1) {
    if (tid == 0) table[0] = make_int4(8 * longest, 0, 0, 0);
    for (int x = wave; x < 8; x += NT / 64)
      for (int i = run(x + 1) - run(x) + lane; i < longest; i += 64) table[1 + 8 * i + x] = make_int4(0, 0, 0, 0);
  }
  // a wave per group and run
  for (int item = part * (NT / 64) + wave; item < 8 * (G + 1); item += parts * (NT / 64)) {
    const int g = item >> 3, x = item & 7, run0 = run(x), run1 = run(x + 1);
    const int p0 = max(first[g] * tiles_n, run0), p1 = min(first[g + 1] * tiles_n, run1);
    if (p0 >= p1) continue;
    const int n = first[g + 1] - first[g], c = cost[g + 1] - cost[g];
    int before = 0;  // the products of the run's groups that come first
    for (int h = lane; h <= G; h += 64) {
      const int products = min(first[h + 1] * tiles_n, run1) - max(first[h] * tiles_n, run0);
      const int64_t mine = static_cast<int64_t>(c) * (first[h + 1] - first[h]);
      const int64_t its = static_cast<int64_t>(cost[h + 1] - cost[h]) * n;
      if (products > 0 && (its > mine || (its == mine && h < g))) before += products;
    }
    before = __builtin_amdgcn_readlane(wave_prefix_sum(before), 63);
    const int row0 = start[g], end = start[g + 1];
    for (int p = p0 + lane; p < p1; p += 64) {
      int tm, tn;
      group_product(p - first[g] * tiles_n, n, tiles_n, tm, tn);
      const int row = row0 + tm * rows;
      table[1 + 8 * (before + p - p0) + x] = make_int4(g < G ? g : -1, row, min(rows, end - row), tn);
    }
  }
}

}  // namespace i8mm
