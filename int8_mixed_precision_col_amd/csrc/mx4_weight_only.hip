// Weight-only MX4 product for at most 16 tokens: Y = X W4^T with 16-bit X (fp16 or bf16),
// fp32 accumulation, one rounding.
//
// One workgroup per 16 output features; its waves share the quads of K and their partial
// sums meet in LDS (weight_stream.hpp has the arithmetic of a quad).
#include "mx4_launch.hpp"
#include "weight_stream.hpp"

namespace i8mm {

constexpr int kMxWoWaves = 8;

template <class T>
__global__ __launch_bounds__(64 * kMxWoWaves) void k_mx_weight_only(MxWeightOnlyArgs a) {
  __shared__ float red[kMxWoWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tok = lane & 15;
  const int ks = mx_ks(a.K), quads = mx_quads(a.K);
  // rows past M and elements past K are out of the resource's range and read zeros
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, static_cast<unsigned>(((a.M - 1) * a.ldx + a.K) * 2));
  const unsigned row = static_cast<unsigned>(tok * a.ldx);
  v4f acc = {};
  for (int q = wave; q < quads; q += kMxWoWaves) {
    WeightQuad<true> w;
    ActQuad<true> x;
    w.load(a.Wc, a.Ws, blockIdx.x, ks, quads, q, lane);
    x.load(q, lane, [&](int k) { return buf_load16(xr, tok < a.M && k < a.K ? (row + k) * 2u : kOOB); });
    mma_quad<T, true>(x, w, acc);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][4 * (lane >> 4) + e][tok] = acc[e];
  lds_barrier();
  const int m = tid >> 4, nl = tid & 15;
  if (m < a.M) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kMxWoWaves; ++w) s += red[w][m][nl];
    static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(m) * a.N + blockIdx.x * 16 + nl] = T::round(s);
  }
}

hipError_t launch_mx_weight_only(const MxWeightOnlyArgs& a, int type, hipStream_t s) {
  const dim3 grid(a.N / 16);
  if (type == kMxF16) hipLaunchKernelGGL(k_mx_weight_only<F16>, grid, dim3(64 * kMxWoWaves), 0, s, a);
  else hipLaunchKernelGGL(k_mx_weight_only<B16>, grid, dim3(64 * kMxWoWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace i8mm
