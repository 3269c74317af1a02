// C ABI of the operators whose rows have weights of their own: argument validation, workspace
// layout, dispatch. Declarations and the contract of each call are in include/groupmm.h.
#include <math.h>
#include <stdint.h>

#include "group.hpp"
#include "group_launch.hpp"
#include "groupmm.h"
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace {

constexpr int64_t kMaxK = int64_t(1) << 20;
constexpr int64_t kMaxInt8K = 133144;  // the int8 operators' own limit
constexpr int64_t kMaxMN = int64_t(1) << 24;
constexpr int64_t kMaxElements = int64_t(1) << 36;
constexpr int64_t kMaxOffset = int64_t(1) << 32;  // bytes a lane's 32-bit offset reaches
constexpr int64_t kMaxRank = 128;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool bad_k(int64_t K) { return K < 16 || K % 16 != 0 || K > kMaxK; }
bool bad_n(int64_t N) { return N < 16 || N % 16 != 0 || N > kMaxMN; }
bool bad_m(int64_t M) { return M < 1 || M > kMaxMN; }
bool bad_ld(int64_t ld, int64_t K) { return ld < K || ld % 8 != 0 || ld > kMaxElements; }
bool bad_dtype16(int t) { return t != MX4_F16 && t != MX4_BF16; }
bool too_many(int64_t rows, int64_t K) { return rows > kMaxElements / K; }
bool bad_top_k(int64_t k) { return k < 1 || k > i8mm::kMoeMaxTopK; }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int hip_status(hipError_t e) { return e == hipSuccess ? INT8MM_OK : INT8MM_E_HIP; }

bool bad_route(int64_t T, int64_t E) { return bad_m(T) || E < 1 || E > i8mm::kMoeMaxExperts; }

bool bad_grouped(int64_t M, int64_t K, int64_t P, int64_t E, int64_t N, int format, int64_t max_outliers) {
  if (bad_m(M) || bad_k(K) || bad_m(P) || E < 1 || E > i8mm::kMaxGroupsOfRows || bad_n(N) || N > kMaxMN / E ||
      too_many(M, K) || too_many(E * N, K) || too_many(P, N) || (format != 0 && format != 1))
    return true;
  if (format == 0)
    return K > kMaxInt8K || int8_quant_state_bytes(M, K, max_outliers) == 0;
  const int64_t row = int64_t(i8mm::mx_ks(K)) * i8mm::kUnitK;
  return (M + 1) * row >= kMaxOffset || N * row >= kMaxOffset;
}

// What X is quantized to and, MX4, the order of the products.
struct GroupedLayout {
  i8mm::GroupTile tile;
  int tiles_n, tiles_most, capacity;
  size_t scales = 0, table = 0, total = 0;
};
GroupedLayout grouped_layout(int64_t M, int64_t K, int64_t P, int64_t E, int64_t N, int format, int64_t max_outliers) {
  GroupedLayout L;
  L.tile = i8mm::pick_group_tile(P, E, N, K, format == 0);
  const int64_t features = i8mm::group_tile_features(L.tile);
  L.tiles_n = int((N + features - 1) / features);
  L.tiles_most = int(i8mm::group_tiles_most(P, E, i8mm::group_tile_rows(L.tile)));
  L.capacity = (L.tiles_n * L.tiles_most + 7) / 8 * 8;  // eight equal runs
  if (format == 0) {
    L.total = round256(int8_quant_state_bytes(M, K, max_outliers));
  } else {
    L.scales = round256(size_t(M + 1) * i8mm::mx_ks(K) * i8mm::kUnitK);
    L.table = L.scales + round256(size_t(M + 1) * i8mm::mx_quads(K) * 16);
    L.total = L.table + round256((1 + size_t(L.capacity)) * sizeof(int4));
  }
  return L;
}

bool bad_lora(int64_t M, int64_t K, int64_t S, int64_t R) {
  return bad_m(M) || bad_k(K) || too_many(M, K) || S < 1 || S > i8mm::kMaxGroupsOfRows || R < 8 || R % 8 != 0 ||
         R > kMaxRank;
}

struct LoraLayout {
  size_t table = 0, part = 0, total = 0;
  int splits = 1;
};
LoraLayout lora_layout(int64_t M, int64_t K, int64_t S, int64_t R) {
  LoraLayout L;
  L.splits = i8mm::lora_splits(M, K, S);
  L.table = round256(size_t(M) * 4);
  L.part = L.table + round256(size_t(1 + i8mm::group_tiles_most(M, S, i8mm::kLoraRows)) * sizeof(int4));
  L.total = L.part + round256(size_t(L.splits) * M * ((R + 15) / 16 * 16) * 4);
  return L;
}

}  // namespace

extern "C" {

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
  return bad_route(T, E) ? 0 : round256(i8mm::route_scratch_bytes(T, E));
}

int moe_route(const void* logits, int64_t T, int64_t E, int logits_dtype, int64_t top_k, int renormalize, int32_t* ids,
              float* weights, int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace, size_t workspace_bytes,
              hipStream_t stream) {
  if (!logits || !ids || !weights || !offsets || !rows || !slots) return INT8MM_E_NULL;
  if (bad_route(T, E) || bad_top_k(top_k) || top_k > E || logits_dtype < MX4_F16 || logits_dtype > MX4_F32)
    return INT8MM_E_SHAPE;
  const size_t need = moe_route_workspace_bytes(T, E);
  if (need && !workspace) return INT8MM_E_NULL;
  if (!aligned16(logits) || !aligned4(ids) || !aligned4(weights) || !aligned4(offsets) || !aligned4(rows) ||
      !aligned4(slots) || !aligned16(workspace))
    return INT8MM_E_ALIGN;
  if (workspace_bytes < need) return INT8MM_E_WORKSPACE;
  const i8mm::RouteArgs a{logits, int(T), int(E), int(top_k), logits_dtype, renormalize != 0, ids, weights, offsets,
                          rows, slots, static_cast<int32_t*>(workspace)};
  return hip_status(i8mm::launch_route(a, stream));
}

size_t moe_grouped_workspace_bytes(int64_t M, int64_t K, int64_t P, int64_t E, int64_t N, int weight_format,
                                   int64_t max_outliers) {
  return bad_grouped(M, K, P, E, N, weight_format, max_outliers)
             ? 0
             : grouped_layout(M, K, P, E, N, weight_format, max_outliers).total;
}

int moe_grouped_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, int weight_format, const void* w,
                       const void* s, int64_t E, int64_t N, const int32_t* offsets, const int32_t* rows, int64_t P,
                       int gated, float threshold, int64_t max_outliers, void* Y, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  if (!X || !w || !s || !offsets || !Y || !workspace) return INT8MM_E_NULL;
  if (bad_grouped(M, K, P, E, N, weight_format, max_outliers) || bad_ld(ldx, K) || bad_dtype16(dtype) ||
      (!rows && P != M) || (gated && N % 32 != 0))
    return INT8MM_E_SHAPE;
  if (weight_format == 0 && (dtype != MX4_F16 || (ldx != K && M > 1))) return INT8MM_E_SHAPE;
  if (weight_format == 0 && (isnan(threshold) || threshold < 0.0f)) return INT8MM_E_THRESHOLD;
  if (!aligned16(X) || !aligned16(w) || !aligned16(s) || !aligned4(offsets) || !aligned4(rows) || !aligned16(Y) ||
      !aligned16(workspace))
    return INT8MM_E_ALIGN;
  const GroupedLayout L = grouped_layout(M, K, P, E, N, weight_format, max_outliers);
  if (workspace_bytes < L.total) return INT8MM_E_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  i8mm::GroupShape shape{int(M), int(K), int(N), int(P), gated != 0, rows, offsets, int(E), L.tiles_most, nullptr, Y};
  if (weight_format == 0) {
    char* st = ws;
    int rc = int8_quantize_activations(X, M, K, threshold, max_outliers, st, workspace_bytes, stream);
    if (rc != INT8MM_OK) return rc;
    int64_t at[6];
    rc = int8_quant_state_layout(M, K, max_outliers, at);
    if (rc != INT8MM_OK) return rc;
    i8mm::Int8GroupArgs a{shape, {}};
    a.q.Wq = static_cast<const int8_t*>(w);
    a.q.a_w = static_cast<const float*>(s);
    a.q.M = int(M); a.q.N = int(N); a.q.K = int(K);
    a.q.a_x = reinterpret_cast<const float*>(st + at[0]);
    a.q.Xq = reinterpret_cast<const int8_t*>(st + at[1]);
    a.q.Xo = reinterpret_cast<const _Float16*>(st + at[2]);
    a.q.idx = reinterpret_cast<const int32_t*>(st + at[3]);
    a.q.count = reinterpret_cast<const int32_t*>(st + at[4]);
    a.q.o_stride = int(at[5]);
    a.q.max_outliers = int(max_outliers);
    return hip_status(i8mm::launch_int8_grouped(a, L.tile, stream));
  }
  uint8_t* codes = reinterpret_cast<uint8_t*>(ws);
  uint8_t* scales = reinterpret_cast<uint8_t*>(ws + L.scales);
  int4* table = reinterpret_cast<int4*>(ws + L.table);
  const i8mm::GroupQuantArgs q{X, ldx, int(M), int(K), codes, scales, offsets, int(E), int(P),
                               i8mm::group_tile_rows(L.tile), L.tiles_n, L.tiles_most, L.capacity, table};
  const hipError_t e = i8mm::launch_group_quantize(q, dtype, stream);
  if (e != hipSuccess) return INT8MM_E_HIP;
  shape.table = table;
  const i8mm::MxGroupArgs a{shape, codes, scales, static_cast<const uint8_t*>(w), static_cast<const uint32_t*>(s),
                             L.capacity};
  return hip_status(i8mm::launch_mx_grouped(a, L.tile, dtype, stream));
}

int moe_combine(const void* P, int64_t P_rows, int64_t D, int dtype, const int32_t* slots, const float* weights,
                int64_t T, int64_t top_k, void* Y, hipStream_t stream) {
  if (!P || !slots || !weights || !Y) return INT8MM_E_NULL;
  if (P_rows < 1 || P_rows > kMaxMN * i8mm::kMoeMaxTopK || bad_k(D) || bad_m(T) || too_many(P_rows, D) ||
      too_many(T, D) || bad_top_k(top_k) || bad_dtype16(dtype))
    return INT8MM_E_SHAPE;
  if (!aligned16(P) || !aligned4(slots) || !aligned4(weights) || !aligned16(Y)) return INT8MM_E_ALIGN;
  const i8mm::CombineArgs a{P, int(T), int(top_k), int(D), P_rows, slots, weights, Y};
  return hip_status(i8mm::launch_combine(a, dtype, stream));
}

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t S, int64_t R) {
  return bad_lora(M, K, S, R) ? 0 : lora_layout(M, K, S, R).total;
}

int lora_apply(const void* Y, int64_t ldy, const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, const void* A,
               const void* B, int64_t S, int64_t R, int64_t N, const int32_t* ids, const float* scales,
               const int32_t* ranks, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
  if (!Y || !X || !A || !B || !ids || !out || !workspace) return INT8MM_E_NULL;
  if (bad_lora(M, K, S, R) || bad_n(N) || too_many(M, N) || too_many(S * R, N) || too_many(S * R, K) ||
      bad_ld(ldx, K) || bad_ld(ldy, N) || bad_ld(ldo, N) || (out == Y && ldo != ldy) || bad_dtype16(dtype))
    return INT8MM_E_SHAPE;
  if (!aligned16(Y) || !aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned4(ids) || !aligned4(scales) ||
      !aligned4(ranks) || !aligned16(out) || !aligned16(workspace))
    return INT8MM_E_ALIGN;
  const LoraLayout L = lora_layout(M, K, S, R);
  if (workspace_bytes < L.total) return INT8MM_E_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const i8mm::LoraArgs a{X, Y, A, B, ldx, ldy, ldo, int(M), int(K), int(N), int(R), int(S), ids, scales, ranks, out,
                         reinterpret_cast<int32_t*>(ws), reinterpret_cast<int4*>(ws + L.table),
                         reinterpret_cast<float*>(ws + L.part), L.splits};
  return hip_status(i8mm::launch_lora(a, dtype, stream));
}

}  // extern "C"
