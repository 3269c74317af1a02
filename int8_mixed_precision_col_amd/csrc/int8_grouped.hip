// The int8 mixed-precision product with a weight per group of rows: for group e and row p of it,
// with x = X[rows[p]],
//   y = (xq Wq_e^T) a_x a_w / 127^2 + sum over outlier columns o of x[o] fp16(Wq_e[., o] a_w / 127),
// the product of gemm_kernel.hpp (which says what each term is), rounded once, or silu(gate) up of
// its two halves. The outlier columns are those of the whole of X.
#include "group_gemm.hpp"
#include "mx4.hpp"

namespace i8mm {

// The epilogue of gemm_kernel.hpp with the rows' constants and outlier values gathered and the
// weight's features by weight_group.
template <class C, bool GATED>
__device__ __forceinline__ void int8_group_epilogue(const Int8GroupArgs& g, const GemmArgs& q, v4i (&acc)[C::BN][C::BM],
                                                    const RowTile& tile, int n0, int wn, int wm, int lane, int tid) {
  constexpr int OS = 24;  // staged row stride in halves (16 columns + 8 of padding)
  static_assert((C::TN + C::TM) * 8 + (C::TN + C::TM) * OS * 2 <= C::STAGE, "staging fits a stage");
  char* base = stage_buf<C, 0>();
  float* aw_s = reinterpret_cast<float*>(base);
  float* ax_s = aw_s + C::TN;
  int* at_s = reinterpret_cast<int*>(ax_s + C::TM);  // feature of the weight, row of X (M: none)
  _Float16* wo_s = reinterpret_cast<_Float16*>(at_s + C::TN + C::TM);
  _Float16* xo_s = wo_s + C::TN * OS;
  const int l16 = lane & 15, lq = lane >> 4;
  const int count = *q.count;
  const bool overflow = count > q.max_outliers;
  const int o_pad = min((count + 15) & ~15, q.o_stride), nvalid = min(count, q.max_outliers);
  const int ks = unit_ks(g.K);
  lds_barrier();  // every wave is done reading the ring
  for (int t = tid; t < C::TN + C::TM; t += C::NT) {
    if (t < C::TN) {
      const int n = weight_group<GATED>(t >> 4, n0, g.N) * 16 + (t & 15);
      at_s[t] = n;
      aw_s[t] = q.a_w[n];
    } else {
      const int m = source_row(g, tile, t - C::TN);
      at_s[t] = m;
      ax_s[t - C::TN] = m < g.M ? q.a_x[m] : 0.0f;
    }
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < C::BN; ++i) {
    const v4f aw = *reinterpret_cast<const v4f*>(aw_s + wn * C::WTN + i * 16 + 4 * lq);
#pragma unroll
    for (int j = 0; j < C::BM; ++j) {
      const float sx = ax_s[wm * C::WTM + j * 16 + l16] * kInvQMax2;
      v4f y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = static_cast<float>(acc[i][j][e]) * sx * aw[e];
      acc[i][j] = __builtin_bit_cast(v4i, y);
    }
  }
  for (int s0 = 0; s0 < o_pad; s0 += 16) {
    if (s0 > 0) lds_barrier();
    for (int t = tid; t < (C::TN + C::TM) * 2; t += C::NT) {
      const int row = t >> 1, h = t & 1, at = at_s[row];
      if (row < C::TN)
        *reinterpret_cast<v8h*>(wo_s + row * OS + 8 * h) = outlier_weights(q, at, s0 + 8 * h, nvalid, ks);
      else
        *reinterpret_cast<v8h*>(xo_s + (row - C::TN) * OS + 8 * h) =
            at < g.M ? *reinterpret_cast<const v8h*>(q.Xo + static_cast<size_t>(at) * q.o_stride + s0 + 8 * h) : v8h{};
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < C::BN; ++i)
#pragma unroll
      for (int j = 0; j < C::BM; ++j) {
        const v4h fa = *reinterpret_cast<const v4h*>(wo_s + (wn * C::WTN + i * 16 + l16) * OS + 4 * lq);
        const v4h fb = *reinterpret_cast<const v4h*>(xo_s + (wm * C::WTM + j * 16 + l16) * OS + 4 * lq);
        acc[i][j] = __builtin_bit_cast(v4i, __builtin_amdgcn_mfma_f32_16x16x16f16(
                                                fa, fb, __builtin_bit_cast(v4f, acc[i][j]), 0, 0, 0));
      }
  }
  lds_barrier();
  store_tile<C, F16, GATED>(g, tile, n0, wn, wm, lane, [&](int i, int j, int e) {
    float v;
    if constexpr (GATED)
      v = silu_up(__builtin_bit_cast(v4f, acc[2 * i][j])[e], __builtin_bit_cast(v4f, acc[2 * i + 1][j])[e]);
    else
      v = __builtin_bit_cast(v4f, acc[i][j])[e];
    return overflow ? __builtin_nanf("") : v;
  });
}

template <class C, bool GATED>
__global__ __launch_bounds__(C::NT) void k_int8_grouped(Int8GroupArgs g, int tiles_n) {
  RowTile tile;
  int tn;
  if (!group_tile_of<C, false>(g, tiles_n, tile, tn)) return;
  const int n0 = tn * (GATED ? C::TN / 2 : C::TN);
  if (tile.group < 0) {
    zero_tile<C, GATED>(g, tile, n0);
    return;
  }
  const int ks = unit_ks(g.K);
  GemmArgs q = g.q;
  q.Wq += static_cast<size_t>(tile.group) * (g.N / 16) * ks * kUnitBytes;
  q.a_w += static_cast<size_t>(tile.group) * g.N;
  GemmBlock<C> b{q};
  const int tid = threadIdx.x, vw = tid >> 6;
  b.lane = tid & 63;
  b.wave = __builtin_amdgcn_readfirstlane(vw);
  b.wn = b.wave % C::WGN;
  b.wm = b.wave / C::WGN;
  b.rn0 = (vw % C::WGN) * C::WTN + (b.lane & 15);
  b.rm0 = (vw / C::WGN) * C::WTM + (b.lane & 15);
#pragma unroll
  for (int i = 0; i < C::AI; ++i) {
    const int p = (i * C::NW + b.wave) * 64 + b.lane, r = p / C::CPR, c = (p % C::CPR) ^ swz<C::CPR>(r);
    b.a_src[i] = q.Wq + unit_offset(weight_group<GATED>(r >> 4, n0, g.N) * 16 + (r & 15), c * 16, ks);
    b.a_k[i] = c * 16;
  }
#pragma unroll
  for (int i = 0; i < C::BI; ++i) {
    const int p = (i * C::NW + b.wave) * 64 + b.lane, r = p / C::CPR, c = (p % C::CPR) ^ swz<C::CPR>(r);
    // rows that are not there take row 0: their constant is 0
    const int m = source_row(g, tile, r);
    b.b_src[i] = q.Xq + unit_offset(m < g.M ? m : 0, c * 16, ks);
    b.b_k[i] = c * 16;
  }
#pragma unroll
  for (int i = 0; i < C::BN; ++i)
#pragma unroll
    for (int j = 0; j < C::BM; ++j) b.acc[i][j] = v4i{};
  const int nk_pad = (ks + C::STAGES - 1) / C::STAGES * C::STAGES;  // slabs past K are zeros
  b.template issue<0>(0);
  b.template issue<1>(1);
  b.template issue<2>(2);
  b.template issue<3>(3);
  typename GemmBlock<C>::Frags f;
  wait_and_barrier<(C::STAGES - 1) * (C::AI + C::BI)>();  // slab 0 landed
  b.template load_frags<0>(f);
  for (int kt = 0; kt < nk_pad; kt += C::STAGES) {
    b.template step<0>(kt, f);
    b.template step<1>(kt + 1, f);
    b.template step<2>(kt + 2, f);
    b.template step<3>(kt + 3, f);
  }
  // no DMA may still be writing this block's LDS when it is reused or the block exits
  __builtin_amdgcn_s_waitcnt(0);
  int8_group_epilogue<C, GATED>(g, q, b.acc, tile, n0, b.wn, b.wm, b.lane, tid);
}

template <class C, bool GATED>
static hipError_t run(const Int8GroupArgs& g, hipStream_t s) {
  constexpr int OUT = GATED ? C::TN / 2 : C::TN;
  const int tiles_n = ((GATED ? g.N / 2 : g.N) + OUT - 1) / OUT;
  hipLaunchKernelGGL((k_int8_grouped<C, GATED>), dim3(static_cast<unsigned>(tiles_n) * g.tiles_most), dim3(C::NT), 0, s,
                     g, tiles_n);
  return hipGetLastError();
}

template <class C>
static hipError_t run(const Int8GroupArgs& g, hipStream_t s) {
  return g.gated ? run<C, true>(g, s) : run<C, false>(g, s);
}

hipError_t launch_int8_grouped(const Int8GroupArgs& g, GroupTile t, hipStream_t s) {
  if (t == GroupTile::L) return run<GroupL>(g, s);
  if (t == GroupTile::S) return run<GroupS>(g, s);
  return run<GroupT>(g, s);
}

}  // namespace i8mm
