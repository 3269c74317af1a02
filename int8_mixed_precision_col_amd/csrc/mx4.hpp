// Microscaled 4-bit ("MX4") operands on gfx950: layout and device helpers.
//
// A row is cut into blocks of 32 consecutive elements. A block holds one power of two
// 2^s, s = clamp(floor(log2 max|x|) - 2, -127, 127), as the byte s + 127, and 32 codes of
// x / 2^s: sign bit 3 and a magnitude index into {0, 0.5, 1, 1.5, 2, 3, 4, 6}, rounded to
// the nearest with ties to the even index and 6 beyond it. A block of zeros has byte 0; a
// block with an infinity or a NaN has byte 255 (every element reads back as NaN) and
// codes 0.
//
// Codes are unit-tiled like the int8 operands: units of 16 rows x 64 bytes, 1 KB
// contiguous, K-fastest within a 16-row group, a unit now covering 128 elements (element
// 2 b of a unit row in the low nibble of byte b). Lane l of a wave that loads its 16 bytes
// of a unit holds row l % 16, elements 32 (l / 16) .. + 31: exactly one block, and exactly
// the 16 x 128 operand of v_mfma_scale_f32_16x16x128_f8f6f4.
// Scale bytes are kept in the order that instruction takes them: per 16-row group and per
// four consecutive units ("quad") 64 dwords, dword l = lane l's block, byte j = unit j of
// the quad. One coalesced 256-byte load gives a wave the scales of four K-steps, and the
// instruction picks the byte. Padding (rows to 16, K to whole quads) is codes 0, byte 0.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace i8mm {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr int kMxUnitK = 128;              // elements of a unit row
constexpr int kMxBlock = 32;               // elements under one scale
__host__ __device__ __forceinline__ int mx_ks(int64_t K) {
  return static_cast<int>((K + kMxUnitK - 1) / kMxUnitK);
}
__host__ __device__ __forceinline__ int mx_quads(int64_t K) { return (mx_ks(K) + 3) >> 2; }

// The scale operand of the conversion instructions for byte b: they read its exponent field
// alone, as a power of two from 2^-127 (field 0) to 2^127, and as NaN for 255 (checked for
// every byte and code).
__device__ __forceinline__ float mx_scale_operand(unsigned b) { return __builtin_bit_cast(float, b << 23); }

// The 16-bit element types: F16 (X, Y fp16) and B16 (bf16).
struct F16 {
  typedef _Float16 elem;
  static constexpr bool bf = false;
  // fp32 exponent field of a magnitude given as its 15 bits (255: not finite)
  static __device__ __forceinline__ unsigned exponent(unsigned mag) {
    const float f = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(mag)));
    return __builtin_bit_cast(unsigned, f) >> 23;
  }
  template <int SEL>
  static __device__ __forceinline__ unsigned to_fp4(unsigned old, unsigned pair, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(v2h, pair), s, SEL);
  }
  template <int SEL>
  static __device__ __forceinline__ unsigned from_fp4(unsigned codes, float s) {
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, SEL));
  }
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ elem round(float v) { return static_cast<_Float16>(v); }
};
struct B16 {
  typedef __bf16 elem;
  static constexpr bool bf = true;
  static __device__ __forceinline__ unsigned exponent(unsigned mag) { return mag >> 7; }
  template <int SEL>
  static __device__ __forceinline__ unsigned to_fp4(unsigned old, unsigned pair, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(v2b, pair), s, SEL);
  }
  template <int SEL>
  static __device__ __forceinline__ unsigned from_fp4(unsigned codes, float s) {
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, SEL));
  }
  static __device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ elem round(float v) { return static_cast<__bf16>(v); }
};

// Largest of the 15-bit magnitudes of 8 elements (as bits: they order like the values, a
// NaN above an infinity above every finite value).
__device__ __forceinline__ unsigned mx_max_bits(const v4u& x) {
  constexpr unsigned m = 0x7fff7fffu;
  const unsigned a = pk_max_u16(pk_max_u16(x[0] & m, x[1] & m), pk_max_u16(x[2] & m, x[3] & m));
  return max(a & 0xffffu, a >> 16);
}

// Scale byte of a block from the fp32 exponent field of its largest magnitude: the field
// less 2, not below 0, and 255 where the block is not finite.
__device__ __forceinline__ unsigned mx_scale_byte(unsigned exponent) {
  return exponent >= 255u ? 255u : exponent >= 2u ? exponent - 2u : 0u;
}

// Codes of 8 elements under scale byte b. The conversion instruction divides by the power of
// two and rounds half-even with saturation at 6. Under 255 the codes mean nothing: what is
// stored has zeros there.
template <class T>
__device__ __forceinline__ unsigned mx_codes8(const v4u& x, unsigned b) {
  const float s = mx_scale_operand(b);
  unsigned c = 0;
  c = T::template to_fp4<0>(c, x[0], s);
  c = T::template to_fp4<1>(c, x[1], s);
  c = T::template to_fp4<2>(c, x[2], s);
  c = T::template to_fp4<3>(c, x[3], s);
  return c;
}

// 8 codes -> 8 elements of T times s.
template <class T>
__device__ __forceinline__ v4u mx_values8(unsigned codes, float s) {
  v4u o;
  o[0] = T::template from_fp4<0>(codes, s);
  o[1] = T::template from_fp4<1>(codes, s);
  o[2] = T::template from_fp4<2>(codes, s);
  o[3] = T::template from_fp4<3>(codes, s);
  return o;
}

// 16x16 tile of W and X codes over one unit, scales from byte SEL of each quad dword:
// D[m = 4 (l / 16) + e][n = l % 16] with x as the first operand.
template <int SEL>
__device__ __forceinline__ v4f mx_mfma(const v4u& a, const v4u& b, const v4f& c, unsigned sa, unsigned sb) {
  const v8i A = {static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3])};
  const v8i B = {static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, SEL, static_cast<int>(sa), SEL,
                                                          static_cast<int>(sb));
}

// Largest value over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (one row's four blocks).
__device__ __forceinline__ unsigned max_over_groups(unsigned v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(static_cast<unsigned>(a[0]), static_cast<unsigned>(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(static_cast<unsigned>(b[0]), static_cast<unsigned>(b[1]));
}

constexpr unsigned kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;  // DPP quad_perm [1,0,3,2], [2,3,0,1]

// Largest value over each aligned group of four lanes.
__device__ __forceinline__ unsigned max_of_four_lanes(unsigned v) {
  v = max(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), kQuadXor1, 0xF, 0xF, true)));
  return max(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), kQuadXor2, 0xF, 0xF, true)));
}

// The wave's own LDS traffic: its writes are done before its later reads, and its reads
// before later writes (other waves have other buffers, so no barrier).
__device__ __forceinline__ void wave_lds_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xF | (0x7 << 4) | (0x0 << 8) | (0x3 << 14));  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

// The lane's number, worked out where it stands rather than held in a register.
__device__ __forceinline__ int lane_again() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// All loads that the wave has asked for are here.
__device__ __forceinline__ void wave_load_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0 | (0x7 << 4) | (0xF << 8));  // vmcnt(0)
  asm volatile("" ::: "memory");
}

}  // namespace i8mm
