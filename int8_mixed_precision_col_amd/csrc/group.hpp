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

// Makes the table of groups 0 .. G - 1 and of the rows behind them, for tiles of tm rows; one
// workgroup of NT threads. Offsets that do not ascend give some table of at most `most` tiles,
// with every row in [0, P).
template <int NT>
__device__ __forceinline__ void make_group_tiles(const int* offsets, int G, int P, int tm, int most, int4* table) {
  __shared__ int first[kMaxGroupsOfRows + 2];  // tiles before group g
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
  const int tiles = min(first[G + 1], most);
  if (tid == 0) table[0] = make_int4(tiles, 0, 0, 0);
  for (int t = tid; t < tiles; t += NT) {
    int lo = 0, hi = G;  // the group g with first[g] <= t < first[g + 1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int row = group_first(offsets, lo, P) + (t - first[lo]) * tm;
    const int end = lo < G ? group_first(offsets, lo + 1, P) : P;
    table[1 + t] = make_int4(lo < G ? lo : -1, row, min(tm, end - row), 0);
  }
}

}  // namespace i8mm
