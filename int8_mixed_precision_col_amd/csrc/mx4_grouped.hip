// Products of MX4 activations with a weight per group of rows: for group e and row p of it,
// Y[p] = MX4(X[rows[p]]) W_e^T, or silu(gate) up of it (products of codes exact, fp32 sums of
// scaled blocks, one rounding).
#include "group_gemm.hpp"
#include "mx4_gemm_kernel.hpp"
#include "mx4_launch.hpp"

#include <algorithm>

namespace i8mm {

template <>
__device__ __forceinline__ char* scale_buf<GroupH>() { return scale_buf<GroupL>(); }

// Rows of X, one after the other, so that the GEMM can take any of them: 64 bytes of codes per
// slab, and 16 bytes of scales per quad (dword b: block b of each unit, byte u: unit u). Lane l of
// a wave holds row l / 16 of four, elements 8 (l % 16) .. + 7 of each unit of a quad. The first
// `parts` workgroups make the table of the products' order meanwhile.
template <class T>
__global__ __launch_bounds__(256) void k_group_quantize(GroupQuantArgs a, int parts) {
  if (static_cast<int>(blockIdx.x) < parts) {
    if (a.tile_rows == GroupL::TM)
      make_balanced_order<256>(a.offsets, a.G, a.P, GroupL::TM, GroupH::TM, a.tiles_n, a.tiles_most, a.capacity, a.table,
                               blockIdx.x, parts);
    else
      make_group_order<256>(a.offsets, a.G, a.P, a.tile_rows, a.tiles_n, a.tiles_most, a.table, blockIdx.x, parts);
    return;
  }
  const int lane = threadIdx.x & 63, r = 4 * (threadIdx.x >> 6) + (lane >> 4), c = lane & 15;
  const int quads = mx_quads(a.K), ks = mx_ks(a.K);
  const int block = blockIdx.x - parts;
  const int64_t grp = block / quads;
  const int q = block - static_cast<int>(grp) * quads;
  const int64_t row = grp * 16 + r;
  const uint16_t* src = static_cast<const uint16_t*>(a.X) + row * a.ldx;
  v4u x[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 512 * q + 128 * u + 8 * c;
    x[u] = v4u{};
    if (row < a.M && k < a.K) x[u] = *reinterpret_cast<const v4u*>(src + k);
  }
  if (row > a.M) return;
  unsigned scale = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const unsigned b = mx_scale_byte(T::exponent(max_of_four_lanes(mx_max_bits(x[u]))));
    scale |= b << (8 * u);
    if (4 * q + u < ks)
      *reinterpret_cast<unsigned*>(a.codes + (row * ks + 4 * q + u) * kUnitK + 4 * c) =
          b == 255u ? 0u : mx_codes8<T>(x[u], b);
  }
  if ((c & 3) == 0) reinterpret_cast<unsigned*>(a.scales)[(row * quads + q) * 4 + (c >> 2)] = scale;
}

hipError_t launch_group_quantize(const GroupQuantArgs& a, int type, hipStream_t s) {
  // a wave per group and run, or an entry of the table per thread, as far as 64 workgroups go
  const int parts = std::min(a.tile_rows == GroupL::TM ? 2 * (a.G + 1) : (a.capacity + 255) / 256, 64);
  const unsigned blocks = static_cast<unsigned>(a.M / 16 + 1) * mx_quads(a.K) + parts;
  if (type == kMxF16) hipLaunchKernelGGL(k_group_quantize<F16>, dim3(blocks), dim3(256), 0, s, a, parts);
  else hipLaunchKernelGGL(k_group_quantize<B16>, dim3(blocks), dim3(256), 0, s, a, parts);
  return hipGetLastError();
}

template <class C, class T, bool GATED>
__device__ __forceinline__ void mx_group_tile(const MxGroupArgs& g, const RowTile& tile, int n0) {
  static_assert(C::STAGES == 4, "a quad of slabs is one turn of the ring");
  typedef MxBlock<C, true> Block;
  Block b;
  const int tid = threadIdx.x, vw = tid >> 6;
  b.lane = tid & 63;
  b.wave = __builtin_amdgcn_readfirstlane(vw);
  const int wn = b.wave % C::WGN, wm = b.wave / C::WGN;
  // per-lane values: as scalars they would hide from the compiler which stage a read touches
  b.rn0 = (vw % C::WGN) * C::WTN + (b.lane & 15);
  b.rm0 = (vw / C::WGN) * C::WTM + (b.lane & 15);
  b.ks = mx_ks(g.K);
  b.quads = mx_quads(g.K);
  const size_t first_group = static_cast<size_t>(tile.group) * (g.N / 16);
  b.a_base = g.Wc + first_group * b.ks * kUnitBytes;
  b.b_base = g.Xc;
  // slot p of a stage holds row p / CPR, chunk (p % CPR) ^ swz(row)
#pragma unroll
  for (int i = 0; i < C::AI; ++i) {
    const int p = (i * C::NW + b.wave) * 64 + b.lane, r = p / C::CPR, c = (p % C::CPR) ^ swz<C::CPR>(r);
    b.a_off[i] = static_cast<unsigned>(weight_group<GATED>(r >> 4, n0, g.N)) * (b.ks * kUnitBytes) + (r & 15) * kUnitK + c * 16;
  }
#pragma unroll
  for (int i = 0; i < C::BI; ++i) {
    const int p = (i * C::NW + b.wave) * 64 + b.lane, r = p / C::CPR, c = (p % C::CPR) ^ swz<C::CPR>(r);
    b.b_off[i] = static_cast<unsigned>(source_row(g, tile, r)) * static_cast<unsigned>(b.ks * kUnitK) + c * 16;
  }
  {
    // scale DMA w: 4 groups of the weight's, 16 lanes each, or 64 rows of X
    static_assert(C::TN % 64 == 0 && C::TM % 64 == 0, "a scale DMA serves one operand");
    const int sw = b.wave % Block::SI, xw = sw - C::TN / 64;
    if (xw < 0) {
      b.s_base = reinterpret_cast<const uint8_t*>(g.Ws) + first_group * b.quads * 256;
      b.s_off = static_cast<unsigned>(weight_group<GATED>(4 * sw + (b.lane >> 4), n0, g.N)) * (b.quads * 256) + 16 * (b.lane & 15);
      b.s_step = 256;
    } else {
      b.s_base = g.Xs;
      b.s_off = static_cast<unsigned>(source_row(g, tile, 64 * xw + b.lane)) * static_cast<unsigned>(b.quads * 16);
      b.s_step = 16;
    }
  }
#pragma unroll
  for (int i = 0; i < C::BN; ++i)
#pragma unroll
    for (int j = 0; j < C::BM; ++j) b.acc[i][j] = v4f{};

  b.issue_scales(0);
  b.template issue<0>(0);
  b.template issue<1>(1);
  b.template issue<2>(2);
  b.template issue<3>(3);
  wait_and_barrier<3 * Block::NQ>();  // scales 0 and slab 0 landed
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
  // a wave whose rows are behind the tile's last only brings its share of the operands
  if (wm * C::WTM < tile.rows) {
    for (int kt = 0; kt < 4 * b.quads; kt += 4) {
      b.template step<0>(kt);
      b.template step<1>(kt + 1);
      b.template step<2>(kt + 2);
      b.template step<3>(kt + 3);
    }
  } else {
    for (int kt = 0; kt < 4 * b.quads; kt += 4) {
      b.template bring<0>(kt);
      b.template bring<1>(kt + 1);
      b.template bring<2>(kt + 2);
      b.template bring<3>(kt + 3);
    }
  }
  // no DMA may still be writing this block's LDS when it is reused or the block exits
  __builtin_amdgcn_s_waitcnt(0);
  lds_barrier();  // every wave is done reading the ring
  store_tile<C, T, GATED>(g, tile, n0, wn, wm, b.lane, [&](int i, int j, int e) {
    if constexpr (GATED) return silu_up(b.acc[2 * i][j][e], b.acc[2 * i + 1][j][e]);
    else return b.acc[i][j][e];
  });
}

template <class C, class T, bool GATED>
__global__ __launch_bounds__(C::NT) void k_mx_grouped(MxGroupArgs g, int tiles_n) {
  RowTile tile;
  int tn;
  if (!group_tile_of<C, true>(g, tiles_n, tile, tn)) return;
  const int n0 = tn * (GATED ? C::TN / 2 : C::TN);
  if (tile.group < 0) {
    zero_tile<C, GATED>(g, tile, n0);
    return;
  }
  if constexpr (C::TM == 256) {
    if (tile.rows <= GroupH::TM) {
      mx_group_tile<GroupH, T, GATED>(g, tile, n0);
      return;
    }
  }
  mx_group_tile<C, T, GATED>(g, tile, n0);
}

template <class C, bool GATED>
static hipError_t run(const MxGroupArgs& g, int type, hipStream_t s) {
  constexpr int OUT = GATED ? C::TN / 2 : C::TN;
  const int tiles_n = ((GATED ? g.N / 2 : g.N) + OUT - 1) / OUT;
  const dim3 grid(g.capacity);
  if (type == kMxF16) hipLaunchKernelGGL((k_mx_grouped<C, F16, GATED>), grid, dim3(C::NT), 0, s, g, tiles_n);
  else hipLaunchKernelGGL((k_mx_grouped<C, B16, GATED>), grid, dim3(C::NT), 0, s, g, tiles_n);
  return hipGetLastError();
}

template <class C>
static hipError_t run(const MxGroupArgs& g, int type, hipStream_t s) {
  return g.gated ? run<C, true>(g, type, s) : run<C, false>(g, type, s);
}

hipError_t launch_mx_grouped(const MxGroupArgs& g, GroupTile t, int type, hipStream_t s) {
  if (t == GroupTile::L) return run<GroupL>(g, type, s);
  return run<GroupT>(g, type, s);
}

}  // namespace i8mm
