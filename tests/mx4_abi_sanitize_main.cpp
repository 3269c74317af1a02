// Host-only driver for the sanitizer build of the MX4 and expert-layer C ABI (no GPU): calls
// that are refused before the library touches the HIP runtime, and the size helpers at the
// int64 limits. Exit status 0 when every return value is the documented one.
#include <stdint.h>
#include <stdio.h>

#include "mx4mm.h"

static int failures = 0;

static void expect(const char* what, long long got, long long want) {
  if (got != want) {
    fprintf(stderr, "FAIL %s: got %lld, want %lld\n", what, got, want);
    ++failures;
  }
}

int main() {
  // fake, 16-byte-aligned device address: never dereferenced, the calls fail first
  void* P = reinterpret_cast<void*>(uintptr_t(0x10000));
  uint8_t* B = static_cast<uint8_t*>(P);
  const int64_t values[] = {INT64_MIN, INT64_MIN + 1, -(int64_t(1) << 40), -1, 0, int64_t(1) << 36, int64_t(1) << 62,
                            INT64_MAX - 7, INT64_MAX};
  for (int64_t v : values) {
    expect("codes rows", mx4_codes_bytes(v, 64), 0);
    expect("codes K", mx4_codes_bytes(64, v), 0);
    expect("scales rows", mx4_scales_bytes(v, 64), 0);
    expect("scales K", mx4_scales_bytes(64, v), 0);
    expect("matmul ws M", mx4_matmul_workspace_bytes(v, 64, 64), 0);
    expect("matmul ws K", mx4_matmul_workspace_bytes(64, v, 64), 0);
    expect("matmul ws N", mx4_matmul_workspace_bytes(64, 64, v), 0);
    expect("q ws M", mx4_matmul_q_workspace_bytes(v, 64, 64), 0);
    expect("q ws K", mx4_matmul_q_workspace_bytes(64, v, 64), 0);
    expect("q ws N", mx4_matmul_q_workspace_bytes(64, 64, v), 0);
    expect("moe ws T", moe_layer_workspace_bytes(v, 64, 2), 0);
    expect("moe ws I", moe_layer_workspace_bytes(4, v, 2), 0);
    expect("moe ws k", moe_layer_workspace_bytes(4, 64, v), 0);
    expect("quantize M", mx4_quantize(P, v, 64, 64, 0, B, B, nullptr), INT8MM_E_SHAPE);
    expect("quantize K", mx4_quantize(P, 4, v, 64, 0, B, B, nullptr), INT8MM_E_SHAPE);
    expect("prepare K", mx4_prepare_weight(P, v, 64, 0, 0, B, B, nullptr), INT8MM_E_SHAPE);
    expect("prepare N", mx4_prepare_weight(P, 64, v, 0, 0, B, B, nullptr), INT8MM_E_SHAPE);
    expect("tile K", mx4_tile_weight(B, B, v, 64, B, B, nullptr), INT8MM_E_SHAPE);
    expect("tile N", mx4_tile_weight(B, B, 64, v, B, B, nullptr), INT8MM_E_SHAPE);
    expect("dequantize M", mx4_dequantize(B, B, v, 64, 0, P, 64, nullptr), INT8MM_E_SHAPE);
    expect("dequantize K", mx4_dequantize(B, B, 4, v, 0, P, 64, nullptr), INT8MM_E_SHAPE);
    expect("matmul M", mx4_matmul(P, v, 64, 64, 0, B, B, 64, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("matmul K", mx4_matmul(P, 4, v, 64, 0, B, B, 64, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("matmul N", mx4_matmul(P, 4, 64, 64, 0, B, B, v, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("matmul_q M", mx4_matmul_q(B, B, v, 64, B, B, 64, 0, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("weight-only M", mx4_weight_only_matmul(P, v, 64, 64, 0, B, B, 64, P, nullptr), INT8MM_E_SHAPE);
    expect("weight-only N", mx4_weight_only_matmul(P, 4, 64, 64, 0, B, B, v, P, nullptr), INT8MM_E_SHAPE);
    expect("moe T", moe_layer(P, v, 64, 64, 0, P, 8, 2, 2, 1, 1, P, P, P, P, 64, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
    expect("moe D", moe_layer(P, 4, v, 64, 0, P, 8, 2, 2, 1, 1, P, P, P, P, 64, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
    expect("moe E", moe_layer(P, 4, 64, 64, 0, P, v, 2, 2, 1, 1, P, P, P, P, 64, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
    expect("moe k", moe_layer(P, 4, 64, 64, 0, P, 8, 2, v, 1, 1, P, P, P, P, 64, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
    expect("moe I", moe_layer(P, 4, 64, 64, 0, P, 8, 2, 2, 1, 1, P, P, P, P, v, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
    if (v < 64 || v % 8 != 0) {  // strides
      expect("quantize ldx", mx4_quantize(P, 4, 64, v, 0, B, B, nullptr), INT8MM_E_SHAPE);
      expect("dequantize ldo", mx4_dequantize(B, B, 4, 64, 0, P, v, nullptr), INT8MM_E_SHAPE);
    }
    if (v != int64_t(1) << 36) continue;
    expect("weight-only ldx", mx4_weight_only_matmul(P, 16, 64, v, 0, B, B, 64, P, nullptr), INT8MM_E_SHAPE);
    expect("matmul ldx", mx4_matmul(P, 16, 64, v, 0, B, B, 64, P, nullptr, 0, nullptr), INT8MM_E_SHAPE);
    expect("moe ldx", moe_layer(P, 16, 64, v, 0, P, 8, 2, 2, 1, 1, P, P, P, P, 64, P, nullptr, nullptr, P, SIZE_MAX, nullptr),
           INT8MM_E_SHAPE);
  }
  // the largest shapes that are taken
  expect("codes largest", static_cast<long long>(mx4_codes_bytes(int64_t(1) << 24, 4096)), int64_t(1) << 35);
  expect("matmul ws few", static_cast<long long>(mx4_matmul_workspace_bytes(16, 4096, 4096)), 0);
  expect("matmul ws 64 rows", static_cast<long long>(mx4_matmul_workspace_bytes(64, 512, 4096)), 0);
  expect("workspace", mx4_matmul(P, 64, 4096, 4096, 0, B, B, 4096, P, P, 1, nullptr), INT8MM_E_WORKSPACE);
  if (failures == 0) printf("all checks passed\n");
  return failures ? 1 : 0;
}
