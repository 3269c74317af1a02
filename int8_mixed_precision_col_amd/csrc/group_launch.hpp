// Host-side launchers of the kernels whose rows have weights of their own (internal to
// libint8mm.so). Each returns hipSuccess or the launch error; arguments are validated by the
// caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace i8mm {

// Routing of T tokens: the chosen experts, and their rows expert after expert.
struct RouteArgs {
  const void* logits;  // [T][E]
  int T, E, k;
  int logits_type;
  int renormalize;
  int32_t* ids;       // [T][k]
  float* weights;     // [T][k]
  int32_t* offsets;   // [E + 1]
  int32_t* rows;      // [T k]
  int32_t* slots;     // [T][k]
  int32_t* counts;    // scratch of route_scratch_bytes(T, E)
};
size_t route_scratch_bytes(int64_t T, int64_t E);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct CombineArgs {
  const void* P;  // [rows][D]
  int T, k, D;
  int64_t rows;
  const int32_t* slots;   // [T][k]
  const float* weights;   // [T][k]
  void* Y;                // [T][D]
};
hipError_t launch_combine(const CombineArgs& a, int type, hipStream_t s);

// Rows of X [M][ldx] to MX4, row by row, and one row M of zeros behind them.
struct GroupQuantArgs {
  const void* X;
  int64_t ldx;
  int M, K;
  uint8_t* codes;   // [M + 1][64 ceil(K / 128)]
  uint8_t* scales;  // [M + 1][16 ceil(K / 512)]: a dword per block of the unit, a byte per unit
  // and, in workgroups of their own, the order of the products (group.hpp)
  const int32_t* offsets;
  int G, P, tile_rows, tiles_n, tiles_most, capacity;
  int4* table;
};
hipError_t launch_group_quantize(const GroupQuantArgs& a, int type, hipStream_t s);

// Shared by both weight formats: P rows, row p of group e (offsets[e] <= p < offsets[e + 1]) against
// that group's N rows of the weight.
struct GroupShape {
  int M, K, N, P;         // rows of X, of K; output features per group; rows of Y
  int gated;              // N is gate features, then as many up features
  const int32_t* rows;    // [P] rows of X, or null: row p
  const int32_t* offsets; // [G + 1]
  int G;
  int tiles_most;         // row tiles that there can be
  const int4* table;      // null, or the order of the products (group.hpp)
  void* Y;                // [P][gated ? N / 2 : N]
};
struct MxGroupArgs : GroupShape {
  const uint8_t *Xc, *Xs;  // GroupQuantArgs
  const uint8_t* Wc;
  const uint32_t* Ws;
  int capacity;           // of the order's table, in workgroups
};
struct Int8GroupArgs : GroupShape {
  GemmArgs q;             // Xq, a_x, Xo, o_stride, idx, count, max_outliers of X; Wq, a_w of all groups
};
// Tile shapes (features x rows): 256 x 256, 128 x 128 (int8 only), 128 x 64.
enum class GroupTile { L, S, T };
int group_tile_rows(GroupTile t);
int group_tile_features(GroupTile t);  // of the weight, gate and up counted
GroupTile pick_group_tile(int64_t P, int64_t groups, int64_t N, int64_t K, bool int8);
hipError_t launch_mx_grouped(const MxGroupArgs& a, GroupTile t, int type, hipStream_t s);
hipError_t launch_int8_grouped(const Int8GroupArgs& a, GroupTile t, hipStream_t s);

// out = Y + scale (X A^T) B^T, each row with its adapter.
struct LoraArgs {
  const void *X, *Y, *A, *B;  // [M][ldx], [M][ldy], [S][R][K], [S][N][R]
  int64_t ldx, ldy, ldo;
  int M, K, N, R, S;
  const int32_t* ids;     // [M]
  const float* scales;    // nullable [S]
  const int32_t* ranks;   // nullable [S]
  void* out;              // [M][ldo]
  int32_t* order;         // scratch: [M] rows by adapter
  int4* table;            // scratch: tiles of kLoraRows rows of `order`
  float* part;            // scratch: [splits][M][16 ceil(R / 16)] sums over parts of K
  int splits;
};
constexpr int kLoraRows = 64;
int lora_splits(int64_t M, int64_t K, int64_t S);
hipError_t launch_lora(const LoraArgs& a, int type, hipStream_t s);

}  // namespace i8mm
