// Weight-only MX4 product for at most 16 tokens: Y = X W4^T with 16-bit X (fp16 or bf16),
// fp32 accumulation, one rounding.
//
// One workgroup per 16 RG output features; its waves share the quads of K and their partial
// sums meet in LDS (weight_stream.hpp has the arithmetic of a quad). Bound by the weight's bytes
// and, for small ones, by launch and first loads: 1 x 12288 x 12288 15.1 us (5.3 TB/s, K x N), 1 x
// 8192 x 8192 8.4 us (4.2 TB/s), 1 x 4096 x 4096 4.2 us.
#include "mx4_launch.hpp"
#include "weight_stream.hpp"

namespace i8mm {

constexpr int kMxWoWaves = 8;

// Waves per SIMD that the registers have to leave room for, 2 of each workgroup: what keeps
// HBM busy is workgroups beside each other on a CU, each waiting for its own loads, and it is
// the rows of X on their way to LDS that take the registers.
constexpr int wo_waves(int rows) { return rows <= 2 ? 6 : rows <= 8 ? 4 : 2; }

// For at most ROWS tokens.
template <class T, int RG, int ROWS>
__global__ __launch_bounds__(64 * kMxWoWaves, wo_waves(ROWS)) void k_mx_weight_only(MxWeightOnlyArgs a) {
  // [waves][act_bytes(M)], and once the products are done the waves' sums: both at a time do
  // not fit for 16 tokens and four row groups
  extern __shared__ __attribute__((aligned(16))) char s_x[];
  float(*red)[16][16 * RG + 1] = reinterpret_cast<float(*)[16][16 * RG + 1]>(s_x);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15;
  const int ks = mx_ks(a.K), quads = mx_quads(a.K), groups = a.N / 16;
  const int g0 = blockIdx.x * RG;
  char* buf = s_x + wave * act_bytes<true>(a.M);
  // what ActQuad leaves out, elements past K among it, is out of the resource's range and reads zeros
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, static_cast<unsigned>(((a.M - 1) * a.ldx + a.K) * 2));
  const int M = a.M, mrow = min(row, M - 1);  // rows past M repeat the last (outputs discarded)
  __builtin_assume(M >= 1 && M <= ROWS);      // the first rows' loads need no test
  // With one row group the wave's next quad is on its way while this one is multiplied (16 x
  // 4096 x 4096 5.4 -> 5.1 us); with more the registers it takes cost more than it gives (16 x
  // 8192 x 8192, two groups: 10.5 -> 11.7 us).
  constexpr bool AHEAD = RG == 1;
  v4f acc[RG] = {};
  WeightQuad<true> w[RG], next[AHEAD ? RG : 1];
  ActQuad<true, ROWS> x;
  auto load_x = [&](int q) {
    // the lane made anew: offsets kept from quad to quad would take the registers that fp16 with 2 rows lacks
    x.load(xr, q, a.K, M, lane_again(), [&](int i) { return static_cast<unsigned>(i * a.ldx) * 2u; });
  };
  auto load_w = [&](auto& to, int q) {
#pragma unroll
    for (int r = 0; r < RG; ++r) to[r].load(a.Wc, a.Ws, min(g0 + r, groups - 1), ks, quads, q, lane);
  };
  if (AHEAD && wave < quads) {
    load_x(wave);
    if constexpr (AHEAD) load_w(next, wave);
  }
  for (int q = wave; q < quads; q += kMxWoWaves) {
    if constexpr (!AHEAD) {
      load_x(q);
      load_w(w, q);
    }
    wave_lds_fence();
    x.store(buf, M, M, lane);
    wave_lds_fence();
    if constexpr (AHEAD) {
#pragma unroll
      for (int r = 0; r < RG; ++r) w[r] = next[r];
      if (q + kMxWoWaves < quads) {
        load_x(q + kMxWoWaves);
        load_w(next, q + kMxWoWaves);
      }
    }
    mma_quad<T, true, RG>(w, acc, [&](int j, int v) { return act_operand<true>(buf, M, mrow, j, v, lane); });
  }
  lds_barrier();  // every wave is done with its rows
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][4 * (lane >> 4) + e][16 * r + row] = acc[r][e];
  lds_barrier();
  for (int o = tid; o < 256 * RG; o += 64 * kMxWoWaves) {
    const int m = o / (16 * RG), n = o % (16 * RG);
    if (m >= M || g0 * 16 + n >= a.N) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kMxWoWaves; ++v) s += red[v][m][n];
    static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(m) * a.N + g0 * 16 + n] = T::round(s);
  }
}

template <int RG, int ROWS>
static hipError_t run_weight_only(const MxWeightOnlyArgs& a, int type, hipStream_t s) {
  const dim3 grid((a.N / 16 + RG - 1) / RG), block(64 * kMxWoWaves);
  const size_t rows = static_cast<size_t>(kMxWoWaves) * act_bytes<true>(a.M);
  const size_t sums = sizeof(float) * kMxWoWaves * 16 * (16 * RG + 1);
  const size_t lds = rows > sums ? rows : sums;
  if (lds > kMaxLds) return hipErrorInvalidConfiguration;
  if (type == kMxF16) hipLaunchKernelGGL((k_mx_weight_only<F16, RG, ROWS>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_mx_weight_only<B16, RG, ROWS>), grid, block, lds, s, a);
  return hipGetLastError();
}

// Row groups per workgroup, by what was measured (us per call, fp16, RG = 1 / 2 / 4, K x N).
hipError_t launch_mx_weight_only(const MxWeightOnlyArgs& a, int type, hipStream_t s) {
  const int groups = a.N / 16;
  // Up to 2 rows three workgroups fit a CU, and one group each is best or near it at any N: M =
  // 2, 4096 x 4096 4.3 / 4.9 / 6.5, 8192 x 8192 8.5 / 8.5 / 10.7, 12288 x 12288 15.1 / 17.4 / 17.0,
  // 2048 x 32768 9.7 / 9.5 / 11.4, 512 x 16384 4.7 / 4.0 / 5.0.
  if (a.M <= 2) return run_weight_only<1, 2>(a, type, s);
  // Up to 8 two do (with 4 groups one): M = 4, 4096 x 4096 4.4 / 5.1 / 7.1, 4096 x 6144 5.4 / 5.5 /
  // 7.4, 8192 x 8192 9.3 / 8.7 / 11.2, 4096 x 10240 7.1 / 7.7 / 7.9, 2048 x 32768 12.2 / 10.1 / 12.7;
  // M = 8, 4096 x 4096 4.8 / 5.4 / 7.3, 4096 x 6144 6.1 / 5.8 / 7.6, 4096 x 10240 7.9 / 8.4 / 8.2.
  if (a.M <= 8) return groups <= 256 ? run_weight_only<1, 8>(a, type, s) : run_weight_only<2, 8>(a, type, s);
  // Beyond that one per CU: as many groups as make one round of workgroups. M = 16, 4096 x 4096
  // 5.3 / 6.1 / 7.9, 4096 x 5120 8.0 / 6.3 / 8.1, 8192 x 8192 14.5 / 10.6 / 12.8, 8192 x 10240 19.9 /
  // 17.2 / 13.6, 4096 x 16384 15.5 / 12.5 / 10.5.
  if (groups <= 256) return run_weight_only<1, 16>(a, type, s);
  return groups <= 512 ? run_weight_only<2, 16>(a, type, s) : run_weight_only<4, 16>(a, type, s);
}

}  // namespace i8mm
