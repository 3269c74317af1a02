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
// multiplied relative to its row's largest block scale, 2^13 for it, and the fp32 sum is scaled
// back. That holds the blocks down to 2^-26 of the largest, as normal numbers; where a row of the
// wave has one below that (trained weights have none, but for blocks of zeros), the quad is gone
// over again for the largest of those. Blocks of byte 0, below 2^-124, are left out of that: no
// fp16 sum can show them beside larger ones.
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

// The activations of one quad of K: loaded whole rows at a time (512 bytes, 256 elements,
// half a wave per row; an MX4 quad has two such pieces), then put through the wave's own LDS
// buffer into operand order. Loading the operand straight from memory takes XV 16-byte
// gathers per unit whatever the number of rows, and those, not the weight, then set the time
// (MX4, 1 x 4096 x 4096: 6.1 us per call; 4.2 so); this takes one load per two rows and piece.
constexpr int kActPiece = 256;                       // elements
constexpr int kActStride = kActPiece * 2 + 16;       // bytes between rows in LDS: a 16-byte
                                                     // skew, so the 16 rows hit distinct banks
template <bool MX, int ROWS>
struct ActQuad {
  static constexpr int P = MX ? 2 : 1;  // pieces of a quad
  v4u raw[P][ROWS / 2];

  // the rows below `rows` (uniform, at most ROWS) of quad q; off(i): row i's byte offset, kOOB
  // for a row of zeros
  template <class F>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int q, int K, int rows, int lane, F off) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int k = (P * q + p) * kActPiece + 8 * (lane & 31);
#pragma unroll
      for (int i = 0; i < ROWS / 2; ++i)
        if (2 * i < rows) {
          const int row = 2 * i + (lane >> 5);
          const unsigned o = row < rows ? off(row) : kOOB;
          raw[p][i] = buf_load16(r, o != kOOB && k < K ? o + 2u * k : kOOB);
        }
    }
  }
  // into LDS: row i of piece p at buf + i * kActStride
  __device__ __forceinline__ void store_piece(int p, char* buf, int rows, int lane) const {
#pragma unroll
    for (int i = 0; i < ROWS / 2; ++i)
      if (2 * i + (lane >> 5) < rows)
        *reinterpret_cast<v4u*>(buf + (2 * i + (lane >> 5)) * kActStride + 16 * (lane & 31)) = raw[p][i];
  }
  // all pieces, `stride` rows each
  __device__ __forceinline__ void store(char* buf, int stride, int rows, int lane) const {
#pragma unroll
    for (int p = 0; p < P; ++p) store_piece(p, buf + p * stride * kActStride, rows, lane);
  }
};
template <bool MX>
__host__ __device__ __forceinline__ constexpr int act_bytes(int rows) {
  return (MX ? 2 : 1) * rows * kActStride;
}

// The operand of unit j (of the quad's 4), 16-byte part v, from rows that ActQuad stored with
// `stride` rows per piece.
template <bool MX>
__device__ __forceinline__ v4u act_operand(const char* buf, int stride, int row, int j, int v, int lane) {
  constexpr int UK = WeightFmt<MX>::UK, KL = WeightFmt<MX>::KL, PER = kActPiece / UK;  // units per piece
  return *reinterpret_cast<const v4u*>(buf + ((j / PER) * stride + row) * kActStride +
                                       2 * (UK * (j % PER) + KL * (lane >> 4) + 8 * v));
}

// The power of two of a row's largest block in fp16 (6 times it is below fp16's largest value) and
// how many below it are still normal numbers with their smallest code, 0.5.
constexpr int kMxTop = 13, kMxWindow = kMxTop + 14 - 1;

// The smallest byte of s that is not 0, less 1 (65535 if all are 0).
__device__ __forceinline__ unsigned mx_least_byte(unsigned s) {
  typedef unsigned short v2s __attribute__((ext_vector_type(2)));
  const v2s one = {1, 1};
  const v2s a = __builtin_bit_cast(v2s, s & 0x00ff00ffu) - one, b = __builtin_bit_cast(v2s, (s >> 8) & 0x00ff00ffu) - one;
  const v2s m = __builtin_elementwise_min(a, b);
  return min(static_cast<unsigned>(m[0]), static_cast<unsigned>(m[1]));
}
// The largest byte of s that is more than kMxWindow below ref (0 if none is).
__device__ __forceinline__ unsigned mx_next_byte(unsigned s, int ref) {
  int most = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b = static_cast<int>((s >> (8 * j)) & 255u);
    if (b + kMxWindow < ref) most = max(most, b);
  }
  return static_cast<unsigned>(most);
}

// What a sum of products relative to block byte ref is multiplied by: NaN for 255, which makes the
// row's outputs NaN whatever else they add up.
__device__ __forceinline__ float mx_back(int ref) {
  return ref == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, ref - 127 - kMxTop);
}

// acc += X_quad W_quad^T in fp16, the blocks by windows of powers of two: of what is left in each row
// (lane l: l % 16) the largest one, ref, and kMxWindow below it. Hardly ever run, and kept small.
template <class T, class X>
__device__ __forceinline__ void mma_quad_spread(const WeightQuad<true>& w, v4f& acc, int ref, X x) {
  for (;;) {
    v4f part = {};
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const int j = i >> 2, v = i & 3;
      v4u unit = w.w[0];
#pragma unroll
      for (int u = 1; u < 4; ++u)
        if (j == u) unit = w.w[u];
      const unsigned codes = v < 2 ? (v ? unit[1] : unit[0]) : (v == 2 ? unit[2] : unit[3]);
      const unsigned b = (w.s >> (8 * j)) & 255u, below = static_cast<unsigned>(ref) - b;
      // 2^-126, so zeros in fp16, for blocks above ref or below the window
      const float s = mx_scale_operand(below <= kMxWindow ? 127 + kMxTop - below : 1u);
      part = T::mfma(x(j, v), mx_values8<T>(codes, s), part);
    }
    const float back = mx_back(ref);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = ref < 0 ? acc[e] : __builtin_fmaf(part[e], back, acc[e]);
    // each turn takes ref down by more than the window; -1: nothing is left of the row
    const int next = static_cast<int>(max_over_groups(mx_next_byte(w.s, ref)));
    ref = next > 0 ? next : -1;
    if (__ballot(ref >= 0) == 0) break;
  }
}

// acc[r] += X_quad W_quad[r]^T for RG row groups of the weight that share the activations
// x(j, v): 16-byte part v of unit j (the int8 column constants are left to the caller).
// J0, J1: of units J0 .. J1 - 1 alone (MX4 in fp16: all four, its reference is theirs).
template <class T, bool MX, int RG, int J0 = 0, int J1 = 4, class X>
__device__ __forceinline__ void mma_quad(const WeightQuad<MX> (&w)[RG], v4f (&acc)[RG], X x) {
  static_assert(!MX || T::bf || J1 - J0 == 4, "the reference of a quad");
  if constexpr (!MX) {
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      const v4u x0 = x(j, 0), x1 = x(j, 1);
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const v2u h0 = int8x4_to16<T>(w[r].w[j][0]), h1 = int8x4_to16<T>(w[r].w[j][1]);
        const v2u h2 = int8x4_to16<T>(w[r].w[j][2]), h3 = int8x4_to16<T>(w[r].w[j][3]);
        acc[r] = T::mfma(x0, v4u{h0[0], h0[1], h1[0], h1[1]}, acc[r]);
        acc[r] = T::mfma(x1, v4u{h2[0], h2[1], h3[0], h3[1]}, acc[r]);
      }
    }
  } else if constexpr (T::bf) {
#pragma unroll
    for (int j = J0; j < J1; ++j) {
      float s[RG];
#pragma unroll
      for (int r = 0; r < RG; ++r) s[r] = mx_scale_operand((w[r].s >> (8 * j)) & 255u);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const v4u xv = x(j, v);
#pragma unroll
        for (int r = 0; r < RG; ++r) acc[r] = T::mfma(xv, mx_values8<T>(w[r].w[j][v], s[r]), acc[r]);
      }
    }
  } else {
    int ref[RG];  // byte of the largest block of lane l's row (l % 16)
    bool spread = false;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const unsigned t = pk_max_u16(w[r].s & 0x00ff00ffu, (w[r].s >> 8) & 0x00ff00ffu);
      ref[r] = static_cast<int>(max_over_groups(max(t & 0xffffu, t >> 16)));
      spread |= static_cast<int>(mx_least_byte(w[r].s)) + 1 + kMxWindow < ref[r];
    }
    if (__builtin_expect(__ballot(spread) == 0, 1)) {
      v4f part[RG] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float s[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const int b = static_cast<int>((w[r].s >> (8 * j)) & 255u);
          s[r] = mx_scale_operand(static_cast<unsigned>(max(127 + kMxTop + b - ref[r], 1)));
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const v4u xv = x(j, v);
#pragma unroll
          for (int r = 0; r < RG; ++r) part[r] = T::mfma(xv, mx_values8<T>(w[r].w[j][v], s[r]), part[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float back = mx_back(ref[r]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = __builtin_fmaf(part[r][e], back, acc[r][e]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < RG; ++r) mma_quad_spread<T>(w[r], acc[r], ref[r], x);
    }
  }
}

}  // namespace i8mm
