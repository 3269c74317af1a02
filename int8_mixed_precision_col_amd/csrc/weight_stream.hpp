// Streaming a quantized weight past 16-bit activations: the part that the MX4 weight-only
// product and the mixture-of-experts kernels share (gfx950).
//
// The unit of work is a quad: four consecutive 1 KB units of one 16-row group of the
// unit-tiled weight (int8: 256 elements of K, MX4: 512). A wave takes whole quads; each
// lane loads its 16 bytes of every unit (row l % 16 of the group, elements KL (l / 16) ..
// of the unit, KL = 16 or 32) and the same elements of its activation row l % 16, turns
// the codes into 16-bit values and feeds them to v_mfma_f32_16x16x32 eight elements at a
// time. Both operands take their K elements from the same lane positions, so the order of
// K inside a unit does not matter. The activations are the first operand: lane l ends with
// D[row 4 (l / 16) + e][feature l % 16].
//
// int8 codes are exact in fp16 and bf16. MX4 values are exact in bf16 (2 significant bits,
// the same exponent range). In fp16 a block's power of two may not fit, so each quad is
// multiplied relative to its row's largest block scale and the fp32 sum is scaled back: a
// value is then inexact only where it is below 2^-23 of the largest power of two of its
// row's quad, off by at most 2^-25 of that.
#pragma once

#include "mx4.hpp"

namespace i8mm {

// 4 int8 codes -> 4 elements of T.
template <class T>
__device__ __forceinline__ v2u int8x4_to16(unsigned d) {
  const unsigned u = d ^ 0x80808080u;  // q + 128 as unsigned bytes
  v2u o;
  if constexpr (!T::bf) {
    // halves 0x64bb = 1024 + b
    const v2h bias = {_Float16(1152.0f), _Float16(1152.0f)};
    o[0] = __builtin_bit_cast(unsigned, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x05010400u)) - bias);
    o[1] = __builtin_bit_cast(unsigned, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, u, 0x05030402u)) - bias);
  } else {
    // fp32 of an integer of at most 8 bits ends in 16 zero bits: its high half is the bf16
    const float f0 = static_cast<float>(u & 255u) - 128.0f, f1 = static_cast<float>((u >> 8) & 255u) - 128.0f;
    const float f2 = static_cast<float>((u >> 16) & 255u) - 128.0f, f3 = static_cast<float>(u >> 24) - 128.0f;
    o[0] = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, f1), __builtin_bit_cast(unsigned, f0), 0x07060302u);
    o[1] = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, f3), __builtin_bit_cast(unsigned, f2), 0x07060302u);
  }
  return o;
}

template <bool MX>
struct WeightFmt {
  static constexpr int UK = MX ? 128 : 64;   // elements of a unit row
  static constexpr int KL = UK / 4;          // elements a lane holds of it
  static constexpr int XV = KL / 8;          // 16-byte activation loads per unit
};

// One quad of one 16-row group in registers.
template <bool MX>
struct WeightQuad {
  v4u w[4];
  unsigned s;  // MX4: the lane's block scales, byte j for unit j

  // group g of a weight with ks units and `quads` quads per group; units past ks reload
  // the last one (their activations are zeros, and MX4 scale bytes past ks are 0)
  __device__ __forceinline__ void load(const void* codes, const uint32_t* scales, size_t g, int ks, int quads,
                                       int q, int lane) {
    const uint8_t* p = static_cast<const uint8_t*>(codes) + g * ks * kUnitBytes + (lane & 15) * kUnitK + 16 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p + static_cast<size_t>(min(4 * q + j, ks - 1)) * kUnitBytes));
    if constexpr (MX) s = scales[(g * quads + q) * 64 + lane];
  }
};

// The activations of one quad: x(k) returns the 8 elements at k .. k + 7 of the lane's row.
template <bool MX>
struct ActQuad {
  v4u x[4][WeightFmt<MX>::XV];
  template <class F>
  __device__ __forceinline__ void load(int q, int lane, F f) {
    constexpr int UK = WeightFmt<MX>::UK, KL = WeightFmt<MX>::KL;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < WeightFmt<MX>::XV; ++v) x[j][v] = f(4 * UK * q + UK * j + KL * (lane >> 4) + 8 * v);
  }
};

// acc += X_quad W_quad^T; the int8 column constant is left to the caller.
template <class T, bool MX>
__device__ __forceinline__ void mma_quad(const ActQuad<MX>& x, const WeightQuad<MX>& w, v4f& acc) {
  if constexpr (!MX) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v2u h0 = int8x4_to16<T>(w.w[j][0]), h1 = int8x4_to16<T>(w.w[j][1]);
      const v2u h2 = int8x4_to16<T>(w.w[j][2]), h3 = int8x4_to16<T>(w.w[j][3]);
      acc = T::mfma(x.x[j][0], v4u{h0[0], h0[1], h1[0], h1[1]}, acc);
      acc = T::mfma(x.x[j][1], v4u{h2[0], h2[1], h3[0], h3[1]}, acc);
    }
  } else if constexpr (T::bf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = mx_scale((w.s >> (8 * j)) & 255u);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc = T::mfma(x.x[j][v], mx_values8<T>(w.w[j][v], s), acc);
    }
  } else {
    const unsigned t = pk_max_u16(w.s & 0x00ff00ffu, (w.s >> 8) & 0x00ff00ffu);
    const unsigned ref = max_over_groups(max(t & 0xffffu, t >> 16));
    v4f part = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned b = (w.s >> (8 * j)) & 255u;
      // 2^(b - ref), at least the smallest normal; NaN for a NaN block
      const float s = mx_scale(b == 255u ? 255u : static_cast<unsigned>(max(static_cast<int>(127 + b - ref), 1)));
#pragma unroll
      for (int v = 0; v < 4; ++v) part = T::mfma(x.x[j][v], mx_values8<T>(w.w[j][v], s), part);
    }
    const float back = mx_scale(ref);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], back, acc[e]);
  }
}

}  // namespace i8mm
