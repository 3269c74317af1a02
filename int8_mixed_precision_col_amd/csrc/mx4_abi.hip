// C ABI of the MX4 and mixture-of-experts operators: argument validation, workspace layout,
// dispatch. Declarations and the contract of each call are in include/mx4mm.h.
#include <stdint.h>

#include "mx4.hpp"
#include "mx4_launch.hpp"
#include "mx4mm.h"

namespace {

constexpr int64_t kMaxK = int64_t(1) << 20;
constexpr int64_t kMaxInt8K = 133144;  // the int8 operators' own limit
constexpr int64_t kMaxMN = int64_t(1) << 24;
constexpr int64_t kMaxElements = int64_t(1) << 36;  // grids stay below 2^32 threads (quantizing 2^24 x 4096: 2^31)
constexpr int64_t kMaxFew = 16;
constexpr int64_t kMaxBuffer = int64_t(1) << 30;    // elements behind a buffer resource

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool bad_k(int64_t K) { return K < 16 || K % 16 != 0 || K > kMaxK; }
bool bad_n(int64_t N) { return N < 16 || N % 16 != 0 || N > kMaxMN; }
bool bad_m(int64_t M) { return M < 1 || M > kMaxMN; }
bool bad_ld(int64_t ld, int64_t K) { return ld < K || ld % 8 != 0 || ld > kMaxElements; }
bool bad_dtype16(int t) { return t != MX4_F16 && t != MX4_BF16; }
bool bad_dtype(int t) { return t < MX4_F16 || t > MX4_F32; }
bool too_many(int64_t rows, int64_t K) { return rows > kMaxElements / K; }

bool bad_product(int64_t M, int64_t K, int64_t N) {
  return bad_m(M) || bad_k(K) || bad_n(N) || too_many(M, K) || too_many(N, K) || too_many(M, N);
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
size_t codes_bytes(int64_t rows, int64_t K) {
  return size_t((rows + 15) / 16) * i8mm::mx_ks(K) * i8mm::kUnitBytes;
}
size_t scales_bytes(int64_t rows, int64_t K) { return size_t((rows + 15) / 16) * i8mm::mx_quads(K) * 256; }
// scratch of the product itself
size_t part_bytes(int64_t M, int64_t K, int64_t N) { return i8mm::mx_few(M) ? 0 : i8mm::mx_gemm_part_bytes(M, N, K); }

int hip_status(hipError_t e) { return e == hipSuccess ? INT8MM_OK : INT8MM_E_HIP; }

hipError_t run_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, uint8_t* codes,
                        void* scales, hipStream_t s) {
  i8mm::MxQuantArgs a{X, ldx, int(M), int(K), codes, static_cast<uint32_t*>(scales)};
  return i8mm::launch_mx_quantize(a, dtype, s);
}

i8mm::MxGemmArgs gemm_args(const uint8_t* xc, const void* xs, int64_t M, int64_t K, const uint8_t* wc,
                           const void* ws, int64_t N, void* Y, void* part) {
  return {xc, static_cast<const uint32_t*>(xs), wc, static_cast<const uint32_t*>(ws), int(M), int(N), int(K),
          Y, int(N), part};
}

hipError_t run_gemm(const i8mm::MxGemmArgs& a, int dtype, hipStream_t s) {
  return i8mm::mx_few(a.M) ? i8mm::launch_mx_few(a, dtype, s) : i8mm::launch_mx_gemm(a, dtype, s);
}

}  // namespace

extern "C" {

size_t mx4_codes_bytes(int64_t rows, int64_t K) {
  return bad_m(rows) || bad_k(K) || too_many(rows, K) ? 0 : codes_bytes(rows, K);
}

size_t mx4_scales_bytes(int64_t rows, int64_t K) {
  return bad_m(rows) || bad_k(K) || too_many(rows, K) ? 0 : scales_bytes(rows, K);
}

int mx4_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, uint8_t* codes,
                 uint8_t* scales, hipStream_t stream) {
  if (!X || !codes || !scales) return INT8MM_E_NULL;
  if (bad_m(M) || bad_k(K) || too_many(M, K) || bad_ld(ldx, K) || bad_dtype16(dtype)) return INT8MM_E_SHAPE;
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scales)) return INT8MM_E_ALIGN;
  return hip_status(run_quantize(X, M, K, ldx, dtype, codes, scales, stream));
}

int mx4_prepare_weight(const void* W, int64_t K, int64_t N, int w_layout, int dtype, uint8_t* codes,
                       uint8_t* scales, hipStream_t stream) {
  if (!W || !codes || !scales) return INT8MM_E_NULL;
  if (bad_k(K) || bad_n(N) || too_many(N, K) || (w_layout != 0 && w_layout != 1) || bad_dtype16(dtype))
    return INT8MM_E_SHAPE;
  if (!aligned16(W) || !aligned16(codes) || !aligned16(scales)) return INT8MM_E_ALIGN;
  if (w_layout == 1) return hip_status(run_quantize(W, N, K, K, dtype, codes, scales, stream));
  return hip_status(i8mm::launch_mx_quantize_cols(W, int(K), int(N), dtype, codes,
                                                  reinterpret_cast<uint32_t*>(scales), stream));
}

int mx4_tile_weight(const uint8_t* packed, const uint8_t* block_scales, int64_t K, int64_t N,
                    uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (!packed || !block_scales || !codes || !scales) return INT8MM_E_NULL;
  if (bad_k(K) || bad_n(N) || too_many(N, K)) return INT8MM_E_SHAPE;
  if (!aligned16(packed) || !aligned16(block_scales) || !aligned16(codes) || !aligned16(scales))
    return INT8MM_E_ALIGN;
  return hip_status(i8mm::launch_mx_tile(packed, block_scales, int(K), int(N), codes,
                                         reinterpret_cast<uint32_t*>(scales), stream));
}

int mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, int dtype,
                   void* out, int64_t ldo, hipStream_t stream) {
  if (!codes || !scales || !out) return INT8MM_E_NULL;
  if (bad_m(M) || bad_k(K) || too_many(M, K) || bad_ld(ldo, K) || bad_dtype(dtype)) return INT8MM_E_SHAPE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return INT8MM_E_ALIGN;
  i8mm::MxDequantArgs a{codes, reinterpret_cast<const uint32_t*>(scales), int(M), int(K), out, ldo};
  return hip_status(i8mm::launch_mx_dequantize(a, dtype, stream));
}

size_t mx4_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (bad_product(M, K, N) || i8mm::mx_few_inline(M, K)) return 0;
  return round256(codes_bytes(M, K)) + round256(scales_bytes(M, K)) + part_bytes(M, K, N);
}

size_t mx4_matmul_q_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return bad_product(M, K, N) ? 0 : part_bytes(M, K, N);
}

int mx4_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, const uint8_t* w_codes,
               const uint8_t* w_scales, int64_t N, void* Y, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
  if (!X || !w_codes || !w_scales || !Y) return INT8MM_E_NULL;
  if (bad_product(M, K, N) || bad_ld(ldx, K) || bad_dtype16(dtype)) return INT8MM_E_SHAPE;
  const bool few = i8mm::mx_few_inline(M, K);
  if (few && M * ldx >= kMaxBuffer) return INT8MM_E_SHAPE;
  if (!few && !workspace) return INT8MM_E_NULL;
  if (!aligned16(X) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y) || !aligned16(workspace))
    return INT8MM_E_ALIGN;
  if (few)
    return hip_status(i8mm::launch_mx_few_inline(gemm_args(nullptr, nullptr, M, K, w_codes, w_scales, N, Y, nullptr), X, ldx,
                                                 dtype, stream));
  if (workspace_bytes < mx4_matmul_workspace_bytes(M, K, N)) return INT8MM_E_WORKSPACE;
  uint8_t* xc = static_cast<uint8_t*>(workspace);
  uint8_t* xs = xc + round256(codes_bytes(M, K));
  const hipError_t e = run_quantize(X, M, K, ldx, dtype, xc, xs, stream);
  if (e != hipSuccess) return INT8MM_E_HIP;
  uint8_t* part = xs + round256(scales_bytes(M, K));
  return hip_status(run_gemm(gemm_args(xc, xs, M, K, w_codes, w_scales, N, Y, part), dtype, stream));
}

int mx4_matmul_q(const uint8_t* x_codes, const uint8_t* x_scales, int64_t M, int64_t K,
                 const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int dtype, void* Y,
                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!x_codes || !x_scales || !w_codes || !w_scales || !Y) return INT8MM_E_NULL;
  if (bad_product(M, K, N) || bad_dtype16(dtype)) return INT8MM_E_SHAPE;
  const size_t need = part_bytes(M, K, N);
  if (need && !workspace) return INT8MM_E_NULL;
  if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y) ||
      !aligned16(workspace))
    return INT8MM_E_ALIGN;
  if (workspace_bytes < need) return INT8MM_E_WORKSPACE;
  return hip_status(run_gemm(gemm_args(x_codes, x_scales, M, K, w_codes, w_scales, N, Y, workspace), dtype, stream));
}

int mx4_weight_only_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype,
                           const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, void* Y,
                           hipStream_t stream) {
  if (!X || !w_codes || !w_scales || !Y) return INT8MM_E_NULL;
  if (M < 1 || M > kMaxFew || bad_k(K) || bad_n(N) || too_many(N, K) || bad_ld(ldx, K) ||
      M * ldx >= kMaxBuffer || bad_dtype16(dtype))
    return INT8MM_E_SHAPE;
  if (!aligned16(X) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(Y)) return INT8MM_E_ALIGN;
  i8mm::MxWeightOnlyArgs a{X, ldx, int(M), int(K), w_codes, reinterpret_cast<const uint32_t*>(w_scales), int(N), Y};
  return hip_status(i8mm::launch_mx_weight_only(a, dtype, stream));
}

size_t moe_layer_workspace_bytes(int64_t T, int64_t I, int64_t top_k) {
  if (T < 1 || T > i8mm::kMoeMaxTokens || bad_k(I) || top_k < 1 || top_k > i8mm::kMoeMaxTopK) return 0;
  return round256(i8mm::moe_workspace(int(T), int(I), int(top_k)));
}

int moe_layer(const void* X, int64_t T, int64_t D, int64_t ldx, int dtype, const void* logits, int64_t E,
              int logits_dtype, int64_t top_k, int renormalize, int weight_format, const void* w13,
              const void* s13, const void* w2, const void* s2, int64_t I, void* Y, int32_t* ids,
              float* weights, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!X || !logits || !w13 || !s13 || !w2 || !s2 || !Y || !workspace) return INT8MM_E_NULL;
  const size_t need = moe_layer_workspace_bytes(T, I, top_k);
  if (need == 0 || bad_k(D) || bad_ld(ldx, D) || T * ldx >= kMaxBuffer || E < 1 || E > i8mm::kMoeMaxExperts ||
      top_k > E || bad_dtype16(dtype) || bad_dtype(logits_dtype) || (weight_format != 0 && weight_format != 1))
    return INT8MM_E_SHAPE;
  if (weight_format == 0 && (D > kMaxInt8K || I > kMaxInt8K)) return INT8MM_E_SHAPE;
  if (!aligned16(X) || !aligned16(logits) || !aligned16(w13) || !aligned16(s13) || !aligned16(w2) ||
      !aligned16(s2) || !aligned16(Y) || !aligned16(ids) || !aligned16(weights) || !aligned16(workspace))
    return INT8MM_E_ALIGN;
  if (workspace_bytes < need) return INT8MM_E_WORKSPACE;
  i8mm::MoeArgs a{X, ldx, int(T), int(D), int(I), int(E), int(top_k), logits, logits_dtype,
                  renormalize != 0, w13, s13, w2, s2, Y, ids, weights, nullptr};
  return hip_status(i8mm::launch_moe(a, workspace, dtype, weight_format == 1, stream));
}

}  // extern "C"
