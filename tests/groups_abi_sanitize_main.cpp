// Host-only driver for the sanitizer build of groupmm.h's C ABI (no GPU): calls that are refused
// before the library touches the HIP runtime, and the size helpers at the int64 limits. Exit
// status 0 when every return value is the documented one.
#include <stdint.h>
#include <stdio.h>

#include "groupmm.h"

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
  void* Q = reinterpret_cast<void*>(uintptr_t(0x20000));
  int32_t* I = static_cast<int32_t*>(P);
  float* F = static_cast<float*>(P);
  const int64_t values[] = {INT64_MIN, INT64_MIN + 1, -(int64_t(1) << 40), -1, 0, int64_t(1) << 36, int64_t(1) << 62,
                            INT64_MAX - 7, INT64_MAX};
  for (int64_t v : values) {
    expect("route ws T", moe_route_workspace_bytes(v, 8), 0);
    expect("route ws E", moe_route_workspace_bytes(100, v), 0);
    for (int format = 0; format < 2; ++format) {
      expect("grouped ws M", moe_grouped_workspace_bytes(v, 64, 8, 4, 32, format, 16), 0);
      expect("grouped ws K", moe_grouped_workspace_bytes(8, v, 8, 4, 32, format, 16), 0);
      expect("grouped ws P", moe_grouped_workspace_bytes(8, 64, v, 4, 32, format, 16), 0);
      expect("grouped ws E", moe_grouped_workspace_bytes(8, 64, 8, v, 32, format, 16), 0);
      expect("grouped ws N", moe_grouped_workspace_bytes(8, 64, 8, 4, v, format, 16), 0);
      expect("grouped M", moe_grouped_matmul(P, v, 64, 64, 0, format, P, P, 4, 32, I, I, 8, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("grouped K", moe_grouped_matmul(P, 8, v, 64, 0, format, P, P, 4, 32, I, I, 8, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("grouped E", moe_grouped_matmul(P, 8, 64, 64, 0, format, P, P, v, 32, I, I, 8, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("grouped N", moe_grouped_matmul(P, 8, 64, 64, 0, format, P, P, 4, v, I, I, 8, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("grouped P", moe_grouped_matmul(P, 8, 64, 64, 0, format, P, P, 4, 32, I, I, v, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    }
    if (v != 0) expect("grouped ws outliers", moe_grouped_workspace_bytes(8, 64, 8, 4, 32, 0, v), 0);
    expect("lora ws M", lora_workspace_bytes(v, 64, 4, 16), 0);
    expect("lora ws K", lora_workspace_bytes(8, v, 4, 16), 0);
    expect("lora ws S", lora_workspace_bytes(8, 64, v, 16), 0);
    expect("lora ws R", lora_workspace_bytes(8, 64, 4, v), 0);
    expect("route T", moe_route(P, v, 8, 2, 2, 1, I, F, I, I, I, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("route E", moe_route(P, 100, v, 2, 2, 1, I, F, I, I, I, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("route k", moe_route(P, 100, 8, 2, v, 1, I, F, I, I, I, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("combine rows", moe_combine(P, v, 64, 0, I, F, 8, 2, P, nullptr), INT8MM_E_SHAPE);
    expect("combine D", moe_combine(P, 8, v, 0, I, F, 8, 2, P, nullptr), INT8MM_E_SHAPE);
    expect("combine T", moe_combine(P, 8, 64, 0, I, F, v, 2, P, nullptr), INT8MM_E_SHAPE);
    expect("combine k", moe_combine(P, 8, 64, 0, I, F, 8, v, P, nullptr), INT8MM_E_SHAPE);
    expect("lora M", lora_apply(P, 32, P, v, 64, 64, 0, P, P, 4, 16, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("lora K", lora_apply(P, 32, P, 8, v, 64, 0, P, P, 4, 16, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("lora S", lora_apply(P, 32, P, 8, 64, 64, 0, P, P, v, 16, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("lora R", lora_apply(P, 32, P, 8, 64, 64, 0, P, P, 4, v, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    expect("lora N", lora_apply(P, 32, P, 8, 64, 64, 0, P, P, 4, 16, v, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    if (v < 64 || v % 8 != 0 || v > (int64_t(1) << 36)) {  // strides
      expect("grouped ldx", moe_grouped_matmul(P, 8, 64, v, 0, 1, P, P, 4, 32, I, I, 8, 0, 6.0f, 16, P, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("lora ldx", lora_apply(P, 32, P, 8, 64, v, 0, P, P, 4, 16, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("lora ldy", lora_apply(P, v, P, 8, 64, 64, 0, P, P, 4, 16, 32, I, F, I, Q, 32, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
      expect("lora ldo", lora_apply(P, 32, P, 8, 64, 64, 0, P, P, 4, 16, 32, I, F, I, Q, v, P, SIZE_MAX, nullptr), INT8MM_E_SHAPE);
    }
  }
  // the largest shapes that are taken
  expect("route largest", moe_route_workspace_bytes(int64_t(1) << 24, 512) > 0, 1);
  expect("grouped largest", moe_grouped_workspace_bytes(1 << 20, 4096, 1 << 24, 1024, 4096, 1, 0) > 0, 1);
  expect("grouped int8 largest", moe_grouped_workspace_bytes(1 << 20, 4096, 1 << 24, 1024, 4096, 0, 4096) > 0, 1);
  expect("lora largest", lora_workspace_bytes(int64_t(1) << 24, 4096, 1024, 128) > 0, 1);
  expect("route workspace", moe_route(P, 100, 8, 2, 2, 1, I, F, I, I, I, P, 1, nullptr), INT8MM_E_WORKSPACE);
  expect("lora workspace", lora_apply(P, 32, P, 8, 64, 64, 0, P, P, 4, 16, 32, I, F, I, Q, 32, P, 1, nullptr), INT8MM_E_WORKSPACE);
  if (failures == 0) printf("all checks passed\n");
  return failures ? 1 : 0;
}
