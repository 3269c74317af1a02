// Product of two MX4 operands: Y [M][N] = X4 W4^T.
//
// Y[m, n] = sum over blocks b of 2^(sx[m, b] + sw[n, b]) sum_{k in b} cx[m, k] cw[n, k], on
// v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies the 4-bit codes, applies both blocks'
// powers of two and accumulates in fp32; one rounding to the output type.
//
// The codes are unit-tiled with 64-byte unit rows like the int8 operands, so the tile walk
// is the int8 GEMM's (gemm_kernel.hpp): slabs of 64 bytes of K, here 128 elements, through
// a ring of LDS stages filled by DMA, one barrier per slab, each DMA instruction a whole
// 1 KB unit. What differs:
//  - Scales. A dword holds a lane's scale bytes of four consecutive units, so they change
//    once per four slabs: the tile's (TN + TM) / 16 groups x 256 bytes of a quad are one
//    more DMA instruction per wave in front of the quad's first slab, into a buffer of
//    their own. It needs no ring: its readers are done one barrier before it is refilled.
//  - Registers. The scales take the registers that a second set of weight fragments would
//    need: a row's fragment (and, at the end of a quad, its scale dword) is read again in
//    place as soon as the row's products are issued, and only the activation side, which
//    every row uses, is held twice.
#include "gemm_kernel.hpp"
#include "gemm_tiles.hpp"
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

#define I8MM_LDS(p) ((__attribute__((address_space(3))) void*)(p))

template <class C>
__device__ __forceinline__ char* scale_buf() {
  __shared__ __attribute__((aligned(1024))) char buf[(C::TN + C::TM) / 16 * 256];
  return buf;
}

template <class C>
struct MxBlock {
  static constexpr int NQ = C::AI + C::BI;              // code DMAs of a wave per slab
  static constexpr int SI = (C::TN + C::TM) / 64;       // scale DMAs of the tile per quad
  static_assert(SI <= C::NW, "one scale DMA per wave");
  const MxGemmArgs& g;
  // uniform bases (the tile's first row groups) and this lane's offsets from them
  const uint8_t *a_base, *b_base, *s_base;
  unsigned a_off[C::AI], b_off[C::BI], s_off;
  int ks, quads;
  int wave, lane, rn0, rm0;
  v4f acc[C::BN][C::BM];
  v4i a[C::BN], b[C::BM];
  unsigned sa[C::BN], sb[C::BM];

  // One DMA instruction (q < AI: weights, else activations) of slab kt into stage S. Slabs
  // past K repeat the last one: those of a last, partial quad are multiplied, but under the
  // layout's padding scales of both sides, 2^-254 together, and add nothing in fp32.
  template <int S>
  __device__ __forceinline__ void issue_one(int kt, int q) {
    const size_t step = static_cast<size_t>(min(kt, ks - 1)) * kUnitBytes;
    char* base = stage_buf<C, S>();
    if (q < C::AI)
      dma16<0>(a_base + step + a_off[q], I8MM_LDS(base + (q * C::NW + wave) * 1024));
    else
      dma16<0>(b_base + step + b_off[q - C::AI], I8MM_LDS(base + C::A_BYTES + ((q - C::AI) * C::NW + wave) * 1024));
  }
  template <int S>
  __device__ __forceinline__ void issue(int kt) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) issue_one<S>(kt, q);
  }
  // The quad's scales. Waves past the last instruction repeat one of them (the same bytes to
  // the same place), so that every wave has the same number of loads in flight.
  __device__ __forceinline__ void issue_scales(int quad) {
    dma16<0>(s_base + static_cast<size_t>(min(quad, quads - 1)) * 256 + s_off,
             I8MM_LDS(scale_buf<C>() + (wave % SI) * 1024));
  }

  template <int S>
  __device__ __forceinline__ v4i frag_a(int i) const {
    return *reinterpret_cast<const v4i*>(stage_buf<C, S>() + lds_off<C::BK>(rn0 + i * 16, lane >> 4));
  }
  template <int S>
  __device__ __forceinline__ v4i frag_b(int j) const {
    return *reinterpret_cast<const v4i*>(stage_buf<C, S>() + C::A_BYTES + lds_off<C::BK>(rm0 + j * 16, lane >> 4));
  }
  // rn0 and rm0 are this lane's rows: their group's dwords start at row / 16
  __device__ __forceinline__ unsigned scale_a(int i) const {
    return reinterpret_cast<const unsigned*>(scale_buf<C>())[((rn0 >> 4) + i) * 64 + lane];
  }
  __device__ __forceinline__ unsigned scale_b(int j) const {
    return reinterpret_cast<const unsigned*>(scale_buf<C>())[(C::TN / 16 + (rm0 >> 4) + j) * 64 + lane];
  }

  template <int SEL>
  static __device__ __forceinline__ v4f mma(const v4i& w, const v4i& x, const v4f& c, unsigned sw, unsigned sx) {
    const v8i A = {w[0], w[1], w[2], w[3]}, B = {x[0], x[1], x[2], x[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, SEL, static_cast<int>(sw), SEL,
                                                            static_cast<int>(sx));
  }

  // Slab kt, whose operands are in registers, with the refill of stage CUR by slab kt + 4
  // (in front of the first slab of a quad its scales) and the reads of slab kt + 1 spread
  // between the products. In flight at the wait, and not waited for: slabs kt + 2 and
  // kt + 3, and the scales issued between them and slab kt + 1.
  template <int CUR>
  __device__ __forceinline__ void step(int kt) {
    constexpr int NX = (CUR + 1) % 4;
    constexpr int EVERY = C::BN * C::BM / NQ > 0 ? C::BN * C::BM / NQ : 1;
    wait_and_barrier<2 * NQ + (CUR == 1 || CUR == 2 ? 1 : 0)>();
    if constexpr (CUR == 0) issue_scales((kt >> 2) + 1);
    v4i nb[C::BM];
    unsigned nsb[C::BM];
#pragma unroll
    for (int j = 0; j < C::BM; ++j) {
      nb[j] = frag_b<NX>(j);
      if constexpr (CUR == 3) nsb[j] = scale_b(j);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < C::BN; ++i) {
#pragma unroll
      for (int j = 0; j < C::BM; ++j) {
        acc[i][j] = mma<CUR>(a[i], b[j], acc[i][j], sa[i], sb[j]);
        const int at = i * C::BM + j;
        if (at % EVERY == EVERY - 1 && at / EVERY < NQ) {
          __builtin_amdgcn_sched_barrier(0);
          issue_one<CUR>(kt + 4, at / EVERY);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      a[i] = frag_a<NX>(i);
      if constexpr (CUR == 3) sa[i] = scale_a(i);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < C::BM; ++j) {
      b[j] = nb[j];
      if constexpr (CUR == 3) sb[j] = nsb[j];
    }
  }
};

// 16x16 accumulator layout: lane l, register e holds row m = l % 16, feature 4 (l / 16) + e.
// Each wave rounds its part of the tile into a slice of the ring and stores whole row
// segments, 16 bytes per lane.
template <class C, class T>
__device__ __forceinline__ void mx_epilogue(const MxGemmArgs& g, v4f (&acc)[C::BN][C::BM], int n0, int m0, int wn,
                                            int wm, int lane) {
  typedef typename T::elem v4t __attribute__((ext_vector_type(4)));
  const int l16 = lane & 15, lq = lane >> 4;
  lds_barrier();  // every wave is done reading the ring
  char* ys = wave_slice<C>(wn + C::WGN * wm);
  constexpr int CH = C::WTN / 8, RB = C::WTN * 2, RPI = 64 / CH;
#pragma unroll
  for (int i = 0; i < C::BN; ++i)
#pragma unroll
    for (int j = 0; j < C::BM; ++j) {
      const int r = j * 16 + l16;
      v4t out;
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = T::round(acc[i][j][e]);
      *reinterpret_cast<v4t*>(ys + r * RB + 16 * ((2 * i + (lane >> 5)) ^ ysw<CH>(r)) + 8 * (lq & 1)) = out;
    }
  const int c = lane % CH;
  const int n = n0 + wn * C::WTN + 8 * c;
#pragma unroll
  for (int t = 0; t < C::WTM / RPI; ++t) {
    const int r = t * RPI + lane / CH;
    const v4u v = *reinterpret_cast<const v4u*>(ys + r * RB + 16 * (c ^ ysw<CH>(r)));
    const int m = m0 + wm * C::WTM + r;
    if (m < g.M && n < g.N)
      *reinterpret_cast<v4u*>(static_cast<uint16_t*>(g.Y) + static_cast<size_t>(m) * g.ldy + n) = v;
  }
}

// The part of K that split s of n takes, in quads: [first, last).
__device__ __forceinline__ void split_range(int quads, int s, int n, int& first, int& last) {
  first = quads * s / n;
  last = quads * (s + 1) / n;
}

// PART: split blockIdx.y of gridDim.y of the K quads, its fp32 sums to g.part in the order of
// the accumulators: [split][tile][wave][i][j][lane] of v4f.
template <class C, class T, bool PART>
__global__ __launch_bounds__(C::NT) void k_mx_gemm(MxGemmArgs g, int tiles_m, int group_m) {
  static_assert(C::STAGES == 4, "a quad of slabs is one turn of the ring");
  int tn, tm;
  tile_of(blockIdx.x, gridDim.x, tiles_m, group_m, tn, tm);
  MxBlock<C> b{g};
  const int tid = threadIdx.x, vw = tid >> 6;
  b.lane = tid & 63;
  b.wave = __builtin_amdgcn_readfirstlane(vw);
  const int wn = b.wave % C::WGN, wm = b.wave / C::WGN;
  // per-lane values: as scalars they would hide from the compiler which stage a read touches
  b.rn0 = (vw % C::WGN) * C::WTN + (b.lane & 15);
  b.rm0 = (vw / C::WGN) * C::WTM + (b.lane & 15);
  b.ks = mx_ks(g.K);
  b.quads = mx_quads(g.K);
  const int n0 = tn * C::TN, m0 = tm * C::TM;
  // slot p of a stage holds row p / CPR, chunk (p % CPR) ^ swz(row); row groups past the
  // edge are clamped (their outputs are discarded)
  const int n_groups = g.N / 16 - n0 / 16, m_groups = (g.M + 15) / 16 - m0 / 16;  // from the tile's first
  b.a_base = g.Wc + static_cast<size_t>(n0 / 16) * b.ks * kUnitBytes;
  b.b_base = g.Xc + static_cast<size_t>(m0 / 16) * b.ks * kUnitBytes;
  auto offset = [&](int p, int groups) {
    const int r = p / C::CPR, c = (p % C::CPR) ^ swz<C::CPR>(r);
    return static_cast<unsigned>(min(r >> 4, groups - 1) * b.ks * kUnitBytes + (r & 15) * kUnitK + c * 16);
  };
#pragma unroll
  for (int i = 0; i < C::AI; ++i) b.a_off[i] = offset((i * C::NW + b.wave) * 64 + b.lane, n_groups);
#pragma unroll
  for (int i = 0; i < C::BI; ++i) b.b_off[i] = offset((i * C::NW + b.wave) * 64 + b.lane, m_groups);
  {
    // scale DMA w: groups 4 w .. 4 w + 3 of the tile (weights first), 16 lanes each
    static_assert(C::TN % 64 == 0, "a scale DMA serves one operand");
    const int sw = b.wave % MxBlock<C>::SI, first = 4 * sw - C::TN / 16;
    const bool w = first < 0;
    b.s_base = reinterpret_cast<const uint8_t*>(w ? g.Ws : g.Xs) +
               static_cast<size_t>(w ? n0 / 16 : m0 / 16) * b.quads * 256;
    const int grp = min((w ? 4 * sw : first) + (b.lane >> 4), (w ? n_groups : m_groups) - 1);
    b.s_off = static_cast<unsigned>(grp * b.quads * 256 + 16 * (b.lane & 15));
  }
#pragma unroll
  for (int i = 0; i < C::BN; ++i)
#pragma unroll
    for (int j = 0; j < C::BM; ++j) b.acc[i][j] = v4f{};

  int q0 = 0, q1 = b.quads;
  if constexpr (PART) split_range(b.quads, blockIdx.y, gridDim.y, q0, q1);
  b.issue_scales(q0);
  b.template issue<0>(4 * q0);
  b.template issue<1>(4 * q0 + 1);
  b.template issue<2>(4 * q0 + 2);
  b.template issue<3>(4 * q0 + 3);
  wait_and_barrier<3 * MxBlock<C>::NQ>();  // scales 0 and slab 0 landed
#pragma unroll
  for (int j = 0; j < C::BM; ++j) {
    b.b[j] = b.template frag_b<0>(j);
    b.sb[j] = b.scale_b(j);
  }
#pragma unroll
  for (int i = 0; i < C::BN; ++i) {
    b.a[i] = b.template frag_a<0>(i);
    b.sa[i] = b.scale_a(i);
  }
  // whole quads: slabs past K are zeros
  for (int kt = 4 * q0; kt < 4 * q1; kt += 4) {
    b.template step<0>(kt);
    b.template step<1>(kt + 1);
    b.template step<2>(kt + 2);
    b.template step<3>(kt + 3);
  }
  // no DMA may still be writing this block's LDS when it is reused or the block exits
  __builtin_amdgcn_s_waitcnt(0);
  if constexpr (PART) {
    v4f* dst = static_cast<v4f*>(g.part) +
               ((static_cast<size_t>(blockIdx.y) * gridDim.x + tn * tiles_m + tm) * C::NW + b.wave) * C::BN * C::BM * 64 +
               b.lane;
#pragma unroll
    for (int i = 0; i < C::BN; ++i)
#pragma unroll
      for (int j = 0; j < C::BM; ++j) dst[(i * C::BM + j) * 64] = b.acc[i][j];
  } else {
    mx_epilogue<C, T>(g, b.acc, n0, m0, wn, wm, b.lane);
  }
}

// Y from the splits' sums, added in order: a wave per accumulator block of a tile.
template <class C, class T>
__global__ __launch_bounds__(256) void k_mx_gemm_join(MxGemmArgs g, int tiles, int tiles_m, int splits) {
  typedef typename T::elem v4t __attribute__((ext_vector_type(4)));
  constexpr int BLOCKS = C::NW * C::BN * C::BM;
  const int lane = threadIdx.x & 63;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 6);  // tile, wave, i, j
  if (at >= tiles * BLOCKS) return;
  const int tile = at / BLOCKS, in = at % BLOCKS;
  const int wave = in / (C::BN * C::BM), i = in / C::BM % C::BN, j = in % C::BM;
  const int n = tile / tiles_m * C::TN + wave % C::WGN * C::WTN + 16 * i + 4 * (lane >> 4);
  const int m = tile % tiles_m * C::TM + wave / C::WGN * C::WTM + 16 * j + (lane & 15);
  if (m >= g.M || n >= g.N) return;
  const v4f* src = static_cast<const v4f*>(g.part) + static_cast<size_t>(at) * 64 + lane;
  v4f sum = src[0];
  for (int s = 1; s < splits; ++s) sum += src[static_cast<size_t>(s) * tiles * BLOCKS * 64];
  v4t out;
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = T::round(sum[e]);
  *reinterpret_cast<v4t*>(static_cast<typename T::elem*>(g.Y) + static_cast<size_t>(m) * g.ldy + n) = out;
}

#undef I8MM_LDS

// 256 x 256, 128 x 256 and 128 x 128 (features x rows) tiles of 8 waves, 4-stage rings.
using MxL = GemmCfg<256, 256, 64, 2, 4, 4>;
using MxM = GemmCfg<128, 256, 64, 2, 4, 4>;
using MxS = GemmCfg<128, 128, 64, 2, 4, 4>;

template <class C>
static hipError_t run(const MxGemmArgs& g, int type, hipStream_t s) {
  const int tiles_n = (g.N + C::TN - 1) / C::TN, tiles_m = (g.M + C::TM - 1) / C::TM;
  const int group_m = tiles_m < 8 ? tiles_m : 8;
  if (type == kMxF16)
    hipLaunchKernelGGL((k_mx_gemm<C, F16, false>), dim3(tiles_n * tiles_m), dim3(C::NT), 0, s, g, tiles_m, group_m);
  else
    hipLaunchKernelGGL((k_mx_gemm<C, B16, false>), dim3(tiles_n * tiles_m), dim3(C::NT), 0, s, g, tiles_m, group_m);
  return hipGetLastError();
}

static hipError_t run_tile(Tile t, const MxGemmArgs& g, int type, hipStream_t s) {
  if (t == Tile::L) return run<MxL>(g, type, s);
  if (t == Tile::M) return run<MxM>(g, type, s);
  return run<MxS>(g, type, s);
}

// Features [n0, n1) as a product of their own (n0 a multiple of 16), into the same rows of Y.
static MxGemmArgs feature_slice(const MxGemmArgs& g, int n0, int n1) {
  MxGemmArgs s = g;
  s.Wc = g.Wc + static_cast<size_t>(n0 / 16) * mx_ks(g.K) * kUnitBytes;
  s.Ws = g.Ws + static_cast<size_t>(n0 / 16) * mx_quads(g.K) * 64;
  s.Y = static_cast<uint16_t*>(g.Y) + n0;
  s.N = n1 - n0;
  return s;
}

static double tile_cost(long M, long N, Tile* t) {
  return best_cost([&](int tn, int tm) { return ((N + tn - 1) / tn) * ((M + tm - 1) / tm); }, t);
}

// The leading features that fill whole waves of 256 x 256 tiles, 0 if that is none or all.
static int whole_wave_features(long M, long N) {
  const long cus = device_cus(), tiles_m = (M + 255) / 256;
  const long n = ((N + 255) / 256) * tiles_m / cus * cus / tiles_m * 256;
  return n < N ? static_cast<int>(n) : 0;
}

template <class C, class T>
static hipError_t run_split(const MxGemmArgs& g, int splits, hipStream_t s) {
  const int tiles_n = (g.N + C::TN - 1) / C::TN, tiles_m = (g.M + C::TM - 1) / C::TM, tiles = tiles_n * tiles_m;
  hipLaunchKernelGGL((k_mx_gemm<C, T, true>), dim3(tiles, splits), dim3(C::NT), 0, s, g, tiles_m,
                     tiles_m < 8 ? tiles_m : 8);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int blocks = tiles * C::NW * C::BN * C::BM;
  hipLaunchKernelGGL((k_mx_gemm_join<C, T>), dim3((blocks + 3) / 4), dim3(256), 0, s, g, tiles, tiles_m, splits);
  return hipGetLastError();
}

// A long K over few tiles leaves most CUs idle while each tile waits for its slabs: K is then
// split, the sums of the splits joined by a second launch. Joining costs 3 to 5 us, so K has at
// least 16 quads (7.5 K elements); more than 192 workgroups write more sums than the split
// saves. Measured, us per product, unsplit against the splits taken here: 128 x 12288 x 4096
// 30.7 / 15.7 (6), 128 x 12288 x 512 22.7 / 11.1 (8), 256 x 8192 x 1024 16.6 / 11.8 (5), 1024 x
// 8192 x 1024 16.8 / 15.0 (3), 128 x 12288 x 12288 33.7 / 26.8 (2); but 128 x 4096 x 4096 10.2 /
// 11.5 (2) and 512 x 12288 x 4096 30.0 / 32.0 (3).
int mx_gemm_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((N + 127) / 128) * ((M + 127) / 128), quads = mx_quads(K);
  if (quads < 16) return 1;
  const int64_t most = quads / 3 < 8 ? quads / 3 : 8, by_tiles = 192 / tiles;
  const int64_t splits = by_tiles < most ? by_tiles : most;
  return splits < 2 ? 1 : static_cast<int>(splits);
}

size_t mx_gemm_part_bytes(int64_t M, int64_t N, int64_t K) {
  const int splits = mx_gemm_splits(M, N, K);
  return splits < 2 ? 0 : static_cast<size_t>(splits) * ((N + 127) / 128) * ((M + 127) / 128) * 128 * 128 * 4;
}

hipError_t launch_mx_gemm(const MxGemmArgs& g, int type, hipStream_t s) {
  const int splits = mx_gemm_splits(g.M, g.N, g.K);
  if (splits > 1) return type == kMxF16 ? run_split<MxS, F16>(g, splits, s) : run_split<MxS, B16>(g, splits, s);
  // Tile shape, and a second launch for the features beyond whole waves of 256 x 256 tiles, by
  // the int8 product's estimate (gemm_tiles.hpp): the tiles' relative rates are within a few
  // percent of its (4096 x 12288 x 49152: 128 x 256 tiles at 0.86 of the 256 x 256 rate, 128 x
  // 128 at 0.80), and it picks the fastest shape or one within 3% of it for 64 to 4096 rows of
  // 1040 x 528 to 12288 x 49152. Two launches: 2048 x 4096 x 11008 56.3 -> 51.2 us.
  Tile t, rest_t;
  const double single = tile_cost(g.M, g.N, &t);
  const int lead = whole_wave_features(g.M, g.N);
  if (lead > 0 && tile_cost(g.M, lead, &rest_t) + tile_cost(g.M, g.N - lead, &rest_t) + 0.05 < single) {
    const hipError_t e = run<MxL>(feature_slice(g, 0, lead), type, s);
    if (e != hipSuccess) return e;
    return run_tile(rest_t, feature_slice(g, lead, g.N), type, s);
  }
  return run_tile(t, g, type, s);
}

}  // namespace i8mm
