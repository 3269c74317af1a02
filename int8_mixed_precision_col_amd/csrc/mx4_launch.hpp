// Host-side launchers of the MX4 and mixture-of-experts kernels (internal to libint8mm.so).
// Each returns hipSuccess or the launch error; arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace i8mm {

// LDS of a workgroup: a launch that asks for more ends the queue, so launchers that size it by
// their arguments check.
constexpr size_t kMaxLds = 160 << 10;

// Element types of the C ABI (mx4_dtype).
enum MxType { kMxF16 = 0, kMxBf16 = 1, kMxF32 = 2 };

// Rows of X [M][ldx] -> codes and scales (mx4.hpp).
struct MxQuantArgs {
  const void* X;
  int64_t ldx;
  int M, K;
  uint8_t* codes;
  uint32_t* scales;
};
hipError_t launch_mx_quantize(const MxQuantArgs& a, int type, hipStream_t s);
// W [K][N] -> codes and scales of the N rows along K.
hipError_t launch_mx_quantize_cols(const void* W, int K, int N, int type, uint8_t* codes,
                                   uint32_t* scales, hipStream_t s);
// Layout only: packed codes [N][16 ceil(K / 32)] and scale bytes [N][ceil(K / 32)].
hipError_t launch_mx_tile(const uint8_t* packed, const uint8_t* bytes, int K, int N,
                          uint8_t* codes, uint32_t* scales, hipStream_t s);
struct MxDequantArgs {
  const uint8_t* codes;
  const uint32_t* scales;
  int M, K;
  void* out;
  int64_t ldo;
};
hipError_t launch_mx_dequantize(const MxDequantArgs& a, int type, hipStream_t s);

// Y [M][N] = X4 W4^T.
struct MxGemmArgs {
  const uint8_t* Xc;
  const uint32_t* Xs;
  const uint8_t* Wc;
  const uint32_t* Ws;
  int M, N, K;
  void* Y;
  int ldy;     // row stride of Y in elements
  void* part;  // mx_gemm_part_bytes(M, N, K) of scratch
};
// Splits of K that a product of few tiles is computed in (1: none), and their fp32 sums' size.
int mx_gemm_splits(int64_t M, int64_t N, int64_t K);
size_t mx_gemm_part_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_gemm(const MxGemmArgs& a, int type, hipStream_t s);
// The same for a few rows: whether it takes them, and the launch. The inline form takes 16-bit
// X itself (a.Xc and a.Xs unused; M ldx < 2^30).
bool mx_few(int64_t M);
hipError_t launch_mx_few(const MxGemmArgs& a, int type, hipStream_t s);
bool mx_few_inline(int64_t M, int64_t K);
hipError_t launch_mx_few_inline(const MxGemmArgs& a, const void* X, int64_t ldx, int type, hipStream_t s);

// Y [M][N] = X W4^T for at most 16 rows of 16-bit X.
struct MxWeightOnlyArgs {
  const void* X;
  int64_t ldx;
  int M, K;
  const uint8_t* Wc;
  const uint32_t* Ws;
  int N;
  void* Y;
};
hipError_t launch_mx_weight_only(const MxWeightOnlyArgs& a, int type, hipStream_t s);

// The mixture-of-experts layer for at most 16 tokens.
constexpr int kMoeMaxTokens = 16, kMoeMaxTopK = 16, kMoeMaxExperts = 512;
struct MoeArgs {
  const void* X;        // [T][ldx]
  int64_t ldx;
  int T, D, I, E, k;
  const void* logits;   // [T][E]
  int logits_type;
  int renormalize;
  const void* w13;      // gate and up rows: E x [gate I rows, up I rows] over D, unit-tiled
  const void* s13;      // int8: fp32 [E 2 I] constants; MX4: scales
  const void* w2;       // down rows: E x D rows over I, unit-tiled
  const void* s2;
  void* Y;              // [T][D]
  int32_t* ids;         // nullable [T][k]
  float* weights;       // nullable [T][k]
  float* h;             // [T k][I]: the hidden rows (set by the launcher)
};
size_t moe_workspace(int T, int I, int k);
hipError_t launch_moe(MoeArgs a, void* workspace, int type, bool mx4, hipStream_t s);

}  // namespace i8mm
