// The K loop of the products of two MX4 operands (mx4_gemm.hip, mx4_grouped.hip): slabs of 64
// bytes of K through a ring of LDS stages, with the scales of four slabs at a time. What it
// does and why is told in mx4_gemm.hip.
#pragma once

#include "gemm_kernel.hpp"
#include "mx4.hpp"

namespace i8mm {

#define I8MM_LDS(p) ((__attribute__((address_space(3))) void*)(p))

template <class C>
__device__ __forceinline__ char* scale_buf() {
  __shared__ __attribute__((aligned(1024))) char buf[(C::TN + C::TM) / 16 * 256];
  return buf;
}

// One workgroup's walk over the slabs of a tile. ROWS: the activations are held row by row, 64
// bytes of codes per slab and 16 of scales per quad, so that a tile's rows can be any rows
// (mx4_grouped.hip); otherwise both operands are unit-tiled.
template <class C, bool ROWS>
struct MxBlock {
  static constexpr int NQ = C::AI + C::BI;              // code DMAs of a wave per slab
  static constexpr int SI = (C::TN + C::TM) / 64;       // scale DMAs of the tile per quad
  static_assert(SI <= C::NW, "one scale DMA per wave");
  // uniform bases (the tile's first row groups) and this lane's offsets from them
  const uint8_t *a_base, *b_base, *s_base;
  unsigned a_off[C::AI], b_off[C::BI], s_off;
  unsigned s_step;  // ROWS: bytes from a quad's scales to the next's, 256 of a weight, 16 of a row
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
      dma16<0>(b_base + (ROWS ? step / kUnitRows : step) + b_off[q - C::AI],
               I8MM_LDS(base + C::A_BYTES + ((q - C::AI) * C::NW + wave) * 1024));
  }
  template <int S>
  __device__ __forceinline__ void issue(int kt) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) issue_one<S>(kt, q);
  }
  // The quad's scales. Waves past the last instruction repeat one of them (the same bytes to
  // the same place), so that every wave has the same number of loads in flight.
  __device__ __forceinline__ void issue_scales(int quad) {
    dma16<0>(s_base + static_cast<size_t>(min(quad, quads - 1)) * (ROWS ? s_step : 256) + s_off,
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
    if constexpr (ROWS)
      return reinterpret_cast<const unsigned*>(scale_buf<C>())[(C::TN + rm0 + j * 16) * 4 + (lane >> 4)];
    return reinterpret_cast<const unsigned*>(scale_buf<C>())[(C::TN / 16 + (rm0 >> 4) + j) * 64 + lane];
  }

  template <int SEL>
  static __device__ __forceinline__ v4f mma(const v4i& w, const v4i& x, const v4f& c, unsigned sw, unsigned sx) {
    const v8i A = {w[0], w[1], w[2], w[3]}, B = {x[0], x[1], x[2], x[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, SEL, static_cast<int>(sw), SEL,
                                                            static_cast<int>(sx));
  }

  // A slab's part of a wave that multiplies nothing: the same waits, barriers and loads.
  template <int CUR>
  __device__ __forceinline__ void bring(int kt) {
    wait_and_barrier<2 * NQ + (CUR == 1 || CUR == 2 ? 1 : 0)>();
    if constexpr (CUR == 0) issue_scales((kt >> 2) + 1);
    issue<CUR>(kt + 4);
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

#undef I8MM_LDS

}  // namespace i8mm
