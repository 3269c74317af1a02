// MX4 product for a few tokens (M <= 64): a weight stream instead of output tiles.
//
// With so few rows the product is bound by reading W4 once from HBM, and 128 x 128 tiles
// would leave most of the GPU idle and multiply padding rows. A workgroup owns 16 RG output
// features and all of M; its waves share the quads of K (four 128-element units each) and
// their fp32 partial sums meet in LDS. Each unit is one operand of
// v_mfma_scale_f32_16x16x128_f8f6f4, straight from global memory to registers.
// With few enough rows X is quantized on the way and the call is one launch: a wave loads a
// row's whole quad at once (1 KB, a lane holds 8 elements and four lanes a block), and the codes
// and scale bytes go through LDS into operand order. Loading 16-bit X in operand order instead
// takes 16 gathers per quad whatever the number of rows (8 x 4096 x 4096: 6.7 us; rows through LDS took it
// to 4.9, and more workgroups per CU to 4.4).
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

constexpr int kFewWaves = 8;
// bytes of a quantized row's quad in LDS: 256 of codes, 16 of scales, and a skew that puts
// the 16 rows of an operand read on distinct banks
constexpr int kFewStride = 256 + 16;

// Where the MX4 activations come from: already tiled; quantized by each wave for the quads it
// multiplies; or all of them quantized by the workgroup's waves together, into LDS.
enum class FewX { kTiled, kOwn, kShared };

// A row's quad, 8 elements per lane, to codes and scale bytes at `to`.
template <class T>
__device__ __forceinline__ void few_quantize(const v4u& x, char* to, int lane) {
  const unsigned b = mx_scale_byte(T::exponent(max_of_four_lanes(mx_max_bits(x))));
  *reinterpret_cast<unsigned*>(to + 4 * lane) = mx_codes8<T>(x, b);
  // block (lane / 4) % 4 of unit lane / 16: byte `unit` of the block's dword
  if ((lane & 3) == 0) to[256 + (lane & 12) + (lane >> 4)] = static_cast<char>(b);
}

// ROWS (kOwn): the most rows; up to 4 leave registers for 6 waves per SIMD, three workgroups
// per CU, which wait for their loads beside each other.
template <class T, int G, int RG, FewX FROM, int ROWS>
__global__ __launch_bounds__(64 * kFewWaves, FROM == FewX::kOwn && ROWS <= 4 ? 6 : 2) void k_mx_few(MxGemmArgs a, const void* X, int64_t ldx) {
  static_assert(FROM != FewX::kOwn || G == 1, "a wave quantizes one row group");
  // rows of kFewStride, then the waves' sums in their place: few_lds()
  extern __shared__ __attribute__((aligned(16))) char s_x[];
  float(*red)[16 * G][16 * RG + 1] = reinterpret_cast<float(*)[16 * G][16 * RG + 1]>(s_x);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15;
  const int ks = mx_ks(a.K), quads = mx_quads(a.K);
  const int groups = a.N / 16, m_groups = (a.M + 15) / 16;
  const int g0 = blockIdx.x * RG;
  const unsigned lane_off = (lane & 15) * kUnitK + 16 * (lane >> 4);

  v4u w[RG][4], x[G][4];
  unsigned ws[RG], xs[G];
  const __amdgpu_buffer_rsrc_t xr =
      make_rsrc(X, FROM != FewX::kTiled ? static_cast<unsigned>(((a.M - 1) * ldx + a.K) * 2) : 0u);
  auto load_row = [&](int m, int q) {  // 8 elements per lane of row m's quad; zeros past K
    const int k = 512 * q + 8 * lane;
    return buf_load16(xr, k < a.K ? static_cast<unsigned>(m * ldx + k) * 2u : kOOB);
  };
  // units past ks repeat the last one, under padding scales (or zeros)
  auto load = [&](int q) {
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const size_t g = min(g0 + r, groups - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[r][j] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(
            a.Wc + (g * ks + min(4 * q + j, ks - 1)) * kUnitBytes + lane_off));
      ws[r] = a.Ws[(g * quads + q) * 64 + lane];
    }
    if constexpr (FROM == FewX::kTiled) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const size_t g = min(i, m_groups - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[i][j] = *reinterpret_cast<const v4u*>(a.Xc + (g * ks + min(4 * q + j, ks - 1)) * kUnitBytes + lane_off);
        xs[i] = a.Xs[(g * quads + q) * 64 + lane];
      }
    }
  };
  if constexpr (FROM == FewX::kShared) {
    // (row, quad) pairs over the waves, four at a time; the first weights are asked for in between
    const int pairs = a.M * quads;
    for (int base = wave; base < pairs; base += 4 * kFewWaves) {
      v4u raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = base + i * kFewWaves;
        if (t < pairs) raw[i] = load_row(t / quads, t % quads);
      }
      if (base == wave && wave < quads) load(wave);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = base + i * kFewWaves;
        if (t < pairs) few_quantize<T>(raw[i], s_x + ((t % quads) * a.M + t / quads) * kFewStride, lane);
      }
    }
    lds_barrier();
  }
  v4f acc[G][RG] = {};
  for (int q = wave; q < quads; q += kFewWaves) {
    v4u raw[FROM == FewX::kOwn ? ROWS : 1];
    if constexpr (FROM == FewX::kOwn) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
        if (i < a.M) raw[i] = load_row(i, q);
    }
    if (FROM != FewX::kShared || q != wave) load(q);
    if constexpr (FROM != FewX::kTiled) {
      const char* rows = s_x + (FROM == FewX::kOwn ? wave * ROWS : q * a.M) * kFewStride;
      if constexpr (FROM == FewX::kOwn) {
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
          if (i < a.M) few_quantize<T>(raw[i], s_x + (wave * ROWS + i) * kFewStride, lane);
        wave_lds_fence();
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const char* p = rows + min(16 * i + row, a.M - 1) * kFewStride;  // rows past M repeat the last
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = *reinterpret_cast<const v4u*>(p + 64 * j + 16 * (lane >> 4));
        xs[i] = *reinterpret_cast<const unsigned*>(p + 256 + 4 * (lane >> 4));
      }
    }
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        acc[i][r] = mx_mfma<0>(x[i][0], w[r][0], acc[i][r], xs[i], ws[r]);
        acc[i][r] = mx_mfma<1>(x[i][1], w[r][1], acc[i][r], xs[i], ws[r]);
        acc[i][r] = mx_mfma<2>(x[i][2], w[r][2], acc[i][r], xs[i], ws[r]);
        acc[i][r] = mx_mfma<3>(x[i][3], w[r][3], acc[i][r], xs[i], ws[r]);
      }
  }
  if constexpr (FROM != FewX::kTiled) lds_barrier();  // every wave is done with the rows
  // lane l, register e: token 4 (l / 16) + e, feature l % 16
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][16 * i + 4 * (lane >> 4) + e][16 * r + row] = acc[i][r][e];
  lds_barrier();
  for (int o = tid; o < 256 * G * RG; o += 64 * kFewWaves) {
    const int m = o / (16 * RG), n = o % (16 * RG);
    if (m >= a.M || g0 * 16 + n >= a.N) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) s += red[v][m][n];
    static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(m) * a.ldy + g0 * 16 + n] = T::round(s);
  }
}

static size_t few_lds(int64_t M, int64_t K, int G, int RG, FewX from, int most) {
  const size_t rows = from == FewX::kTiled ? 0 : from == FewX::kOwn ? kFewWaves * most : mx_quads(K) * M;
  const size_t sums = sizeof(float) * kFewWaves * 16 * G * (16 * RG + 1);
  return rows * kFewStride > sums ? rows * kFewStride : sums;
}

template <int G, int RG, FewX FROM, int ROWS = 16 * G>
static hipError_t run(const MxGemmArgs& a, const void* X, int64_t ldx, int type, hipStream_t s) {
  const dim3 grid((a.N / 16 + RG - 1) / RG), block(64 * kFewWaves);
  const size_t lds = few_lds(a.M, a.K, G, RG, FROM, ROWS);
  if (lds > kMaxLds) return hipErrorInvalidConfiguration;
  if (type == kMxF16) hipLaunchKernelGGL((k_mx_few<F16, G, RG, FROM, ROWS>), grid, block, lds, s, a, X, ldx);
  else hipLaunchKernelGGL((k_mx_few<B16, G, RG, FROM, ROWS>), grid, block, lds, s, a, X, ldx);
  return hipGetLastError();
}

// Row groups per workgroup where each workgroup does much over again that all do (quantizing X, or
// reading 64 rows of it): as many as make one round of workgroups over the CUs, up to 4, although with one
// group two fit a CU (X quantized by each wave for its own quads: 113 registers and 35 KB; two and
// four groups, 136 and 185 registers, one). Measured per call (HIP
// graphs over rotated weights, fp16, K x N, RG = 1 / 2 / 4): M = 16, X quantized on the way, 4096 x
// 4096 6.3 / 6.2 / 7.7 us, 4096 x 6144 8.5 / 6.8 / 7.9, 8192 x 8192 14.8 / 11.5 / 13.2, 4096 x
// 10240 11.6 / 11.3 / 8.6, 12288 x 12288 28.9 / 25.5 / 20.1; M = 64, X tiled, 4096 x 4096 6.2 /
// 7.6 / 8.9, 8192 x 8192 15.2 / 13.6 / 14.7, 4096 x 10240 11.9 / 11.7 / 9.8, 12288 x 12288 30.7 /
// 27.5 / 21.7.
template <int G, FewX FROM>
static hipError_t pick(const MxGemmArgs& a, const void* X, int64_t ldx, int type, hipStream_t s) {
  const int groups = a.N / 16;
  if (groups <= 256) return run<G, 1, FROM>(a, X, ldx, type, s);
  return groups <= 512 ? run<G, 2, FROM>(a, X, ldx, type, s) : run<G, 4, FROM>(a, X, ldx, type, s);
}

// One launch instead of a quantization and a product. Up to 16 rows always; more while the
// workgroup has at most 96 (row, quad) pairs to quantize, which every workgroup does again
// (K x N, one launch against two, us in graphs: 32 rows of 1024 x 1024 5.0 / 5.2, 64 of 512 x 512
// 4.9 / 6.2, 48 of 1024 x 1024 6.3 / 6.2, 24 of 2048 x 4096 6.4 / 5.6; 32 of 2048 x 4096, 128
// pairs, 7.4 / 5.7; outside graphs the second launch costs another 4 us of the caller's time).
bool mx_few_inline(int64_t M, int64_t K) { return M <= 16 || (M <= 64 && M * mx_quads(K) <= 96); }

// Up to 16 rows, by the workgroup together while K has at most two quads, so that six of its
// eight waves do not watch (16 rows of 1024 x 1024 3.5 against 3.9 us, of 2048 x 1024 4.7 against
// 4.4). Up to 4 rows, one group per workgroup and three workgroups per CU, in place of the
// choice above: 4096 x 4096 4.2 against 4.3 us, 4096 x 10240 6.7 / 7.1, 12288 x 12288 16.6 /
// 16.3 (two rows 14.6 / 16.1), 2048 x 32768 9.0 / 10.8, 8192 x 28672 23.3 / 24.8.
hipError_t launch_mx_few_inline(const MxGemmArgs& a, const void* X, int64_t ldx, int type, hipStream_t s) {
  if (a.M <= 16 && mx_quads(a.K) <= 2) return pick<1, FewX::kShared>(a, X, ldx, type, s);
  if (a.M <= 4) return run<1, 1, FewX::kOwn, 4>(a, X, ldx, type, s);
  if (a.M <= 16) return pick<1, FewX::kOwn>(a, X, ldx, type, s);
  return a.M <= 32 ? pick<2, FewX::kShared>(a, X, ldx, type, s) : pick<4, FewX::kShared>(a, X, ldx, type, s);
}

// Up to 64 rows: at 64 the tiles are slower still (4096 x 4096 11.3 against 5.9 us, 4096 x
// 16384 12.7 against 11.2, 8192 x 8192 20.0 against 11.9).
bool mx_few(int64_t M) { return M <= 64; }

// X already tiled takes few registers, so that several workgroups share a CU and one group each
// is best, or near it, until their reading X again shows. RG = 1 / 2 / 4, us: M = 16, 4096 x 4096
// 4.1 / 4.8 / 7.4, 8192 x 8192 9.2 / 8.7 / 13.2, 12288 x 12288 16.9 / 17.9 / 20.6, 8192 x 28672
// 25.7 / 24.5 / 22.9; M = 32, 4096 x 4096 4.6 / 6.1 / 7.8, 8192 x 8192 10.9 / 11.4 / 13.3, 4096 x
// 16384 10.6 / 10.8 / 11.1, 2048 x 32768 11.2 / 10.4 / 10.7, 8192 x 28672 32.8 / 28.8 / 25.0.
hipError_t launch_mx_few(const MxGemmArgs& a, int type, hipStream_t s) {
  if (a.M <= 16) return run<1, 1, FewX::kTiled>(a, nullptr, 0, type, s);
  if (a.M <= 32)
    return a.N < 16 * 1024 ? run<2, 1, FewX::kTiled>(a, nullptr, 0, type, s) : run<2, 4, FewX::kTiled>(a, nullptr, 0, type, s);
  return pick<4, FewX::kTiled>(a, nullptr, 0, type, s);
}

}  // namespace i8mm
