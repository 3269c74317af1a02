// Product of two MX4 operands: Y [M][N] = X4 W4^T.
//
// Y[m, n] = sum over blocks b of 2^(sx[m, b] + sw[n, b]) sum_{k in b} cx[m, k] cw[n, k], on
// v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies the 4-bit codes, applies both blocks'
// powers of two and accumulates in fp32; one rounding to the output type.
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

// A wave per 64 rows x 16 features, operands straight from global memory.
template <class T>
__global__ __launch_bounds__(256) void k_mx_gemm(MxGemmArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ks = mx_ks(a.K), quads = mx_quads(a.K);
  const int ng = blockIdx.x * 4 + wave;
  const int mgroups = (a.M + 15) / 16, mg0 = blockIdx.y * 4;
  if (ng >= a.N / 16) return;
  const uint8_t* wc = a.Wc + static_cast<size_t>(ng) * ks * kUnitBytes + (lane & 15) * kUnitK + 16 * (lane >> 4);
  const uint32_t* ws = a.Ws + static_cast<size_t>(ng) * quads * 64 + lane;
  const uint8_t* xc[4];
  const uint32_t* xs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = min(mg0 + i, mgroups - 1);
    xc[i] = a.Xc + static_cast<size_t>(g) * ks * kUnitBytes + (lane & 15) * kUnitK + 16 * (lane >> 4);
    xs[i] = a.Xs + static_cast<size_t>(g) * quads * 64 + lane;
  }
  v4f acc[4] = {};
  for (int s = 0; s < ks; ++s) {
    const v4u w = *reinterpret_cast<const v4u*>(wc + static_cast<size_t>(s) * kUnitBytes);
    const unsigned sw = ws[(s >> 2) * 64] >> (8 * (s & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4u x = *reinterpret_cast<const v4u*>(xc[i] + static_cast<size_t>(s) * kUnitBytes);
      acc[i] = mx_mfma<0>(x, w, acc[i], xs[i][(s >> 2) * 64] >> (8 * (s & 3)), sw);
    }
  }
  const int n = ng * 16 + (lane & 15);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = (mg0 + i) * 16 + 4 * (lane >> 4) + e;
      if (m < a.M) static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(m) * a.ldy + n] = T::round(acc[i][e]);
    }
}

hipError_t launch_mx_gemm(const MxGemmArgs& a, int type, hipStream_t s) {
  const dim3 grid((a.N / 16 + 3) / 4, (a.M + 63) / 64);
  if (type == kMxF16) hipLaunchKernelGGL(k_mx_gemm<F16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_mx_gemm<B16>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace i8mm
