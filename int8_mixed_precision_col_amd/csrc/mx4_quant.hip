// MX4 quantization, its inverse and the layout conversion (format and layout: mx4.hpp).
//
// All four are bound by HBM: 2 bytes read and 17/32 written per element to quantize, the
// reverse to read back. Measured, 1333 x 20464: quantize 12.0 us, read back 12.1 us, 5.7 TB/s
// each (a large copy: 4.9 TB/s); 8 x 4096: 2.6 us each, launch and one round trip.
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

// One workgroup per 16 rows x 512 elements (one quad), a wave per 4 rows: lane l holds row
// l / 16, elements 8 (l % 16) .. + 7 of each of the quad's four units, so that a wave reads
// 256 contiguous bytes of 4 rows per load and writes 256 contiguous bytes of codes per
// store; four neighbouring lanes share a block.
template <class T>
__global__ __launch_bounds__(256) void k_mx_quantize(MxQuantArgs a) {
  const int lane = threadIdx.x & 63, r = 4 * (threadIdx.x >> 6) + (lane >> 4), c = lane & 15;
  const int quads = mx_quads(a.K), ks = mx_ks(a.K);
  const int64_t grp = blockIdx.x / quads;
  const int q = blockIdx.x - static_cast<int>(grp) * quads;
  const int64_t row = grp * 16 + r;
  const uint16_t* src = static_cast<const uint16_t*>(a.X) + row * a.ldx;
  v4u x[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 512 * q + 128 * u + 8 * c;
    x[u] = v4u{};
    if (row < a.M && k < a.K) x[u] = *reinterpret_cast<const v4u*>(src + k);
  }
  unsigned scale = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const unsigned b = mx_scale_byte(T::exponent(max_of_four_lanes(mx_max_bits(x[u]))));
    scale |= b << (8 * u);
    if (4 * q + u < ks)
      *reinterpret_cast<unsigned*>(a.codes + (grp * ks + 4 * q + u) * kUnitBytes + r * kUnitK + 4 * c) =
          b == 255u ? 0u : mx_codes8<T>(x[u], b);
  }
  if ((c & 3) == 0) a.scales[(grp * quads + q) * 64 + 16 * (c >> 2) + r] = scale;
}

hipError_t launch_mx_quantize(const MxQuantArgs& a, int type, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((a.M + 15) / 16) * mx_quads(a.K);
  if (type == kMxF16) hipLaunchKernelGGL(k_mx_quantize<F16>, dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_mx_quantize<B16>, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// W [K][N], blocks down the columns. A workgroup takes 128 columns x one unit of K: wave g
// takes block g of the unit, lane l columns 2 l and 2 l + 1, so that every load of a wave is 256
// contiguous bytes of one row and a lane holds whole blocks of its columns; the pairs along K
// that the conversion wants are put together with v_perm. 4096 x 16384: 42 us, 4.1 TB/s (a
// workgroup per quad instead of per unit 47 us; 4 or 8 columns per lane 44 and 41 us, but 4.5
// and 5.9 against 3.6 us at 1024 x 1024).
template <class T>
__global__ __launch_bounds__(256) void k_mx_quantize_cols(const uint16_t* W, int K, int N, uint8_t* codes,
                                                          uint8_t* scales) {
  constexpr int COLS = 2;
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int n = blockIdx.x * 128 + COLS * lane, u = blockIdx.y;
  if (n >= N) return;
  const int quads = mx_quads(K), ks = mx_ks(K);
  const int64_t grp = n >> 4;
  const int r = n & 15;
  // the unit's place in its quad; the last unit clears the scales of the quad's padding too
  const int last = u + 1 < ks ? u : u | 3;
  unsigned b[COLS];
  const int k0 = 128 * u + 32 * g;
  unsigned x[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    // K is a multiple of 16: each half block is all there or past the end
    x[e] = k0 + (e & 16) < K ? *reinterpret_cast<const unsigned*>(W + static_cast<int64_t>(k0 + e) * N + n) : 0u;
  }
#pragma unroll
  for (int j = 0; j < COLS; ++j) {
    v4u v[4];
    unsigned top = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        v[p][d] = __builtin_amdgcn_perm(x[8 * p + 2 * d + 1], x[8 * p + 2 * d], j ? 0x07060302u : 0x05040100u);
      top = max(top, mx_max_bits(v[p]));
    }
    b[j] = mx_scale_byte(T::exponent(top));
    v4u o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = b[j] == 255u ? 0u : mx_codes8<T>(v[p], b[j]);
    *reinterpret_cast<v4u*>(codes + (grp * ks + u) * kUnitBytes + (r + j) * kUnitK + 16 * g) = o;
  }
#pragma unroll
  for (int j = 0; j < COLS; ++j) {
    uint8_t* to = scales + ((grp * quads + (u >> 2)) * 64 + 16 * g + r + j) * 4;
    to[u & 3] = static_cast<uint8_t>(b[j]);
    for (int i = u + 1; i <= last; ++i) to[i & 3] = 0;
  }
}

hipError_t launch_mx_quantize_cols(const void* W, int K, int N, int type, uint8_t* codes, uint32_t* scales,
                                   hipStream_t s) {
  const uint16_t* w = static_cast<const uint16_t*>(W);
  uint8_t* sc = reinterpret_cast<uint8_t*>(scales);
  const dim3 grid((N + 127) / 128, mx_ks(K));
  if (type == kMxF16) hipLaunchKernelGGL(k_mx_quantize_cols<F16>, grid, dim3(256), 0, s, w, K, N, codes, sc);
  else hipLaunchKernelGGL(k_mx_quantize_cols<B16>, grid, dim3(256), 0, s, w, K, N, codes, sc);
  return hipGetLastError();
}

// Row-major packed codes and scale bytes -> the tiled layout; same lane mapping as
// k_mx_quantize. Codes past K (the second half of a last, half-full block) become 0. Once per
// checkpoint weight: 12288 x 49152 (K x N) 171 us, 3.7 TB/s read and written, 4096 x 16384 20.7, 4096 x
// 4096 6.0 (a large copy: 4.9 TB/s; a lane moves 4 bytes at a time).
__global__ __launch_bounds__(256) void k_mx_tile(const uint8_t* packed, const uint8_t* bytes, int K,
                                                 uint8_t* codes, uint32_t* scales) {
  const int lane = threadIdx.x & 63, r = 4 * (threadIdx.x >> 6) + (lane >> 4), c = lane & 15;
  const int quads = mx_quads(K), ks = mx_ks(K), nb = (K + kMxBlock - 1) / kMxBlock;
  const int64_t grp = blockIdx.x / quads;
  const int q = blockIdx.x - static_cast<int>(grp) * quads;
  const int64_t row = grp * 16 + r;
  unsigned scale = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 512 * q + 128 * u + 8 * c;
    unsigned v = 0;
    if (k < K) {
      v = *reinterpret_cast<const unsigned*>(packed + row * nb * 16 + k / 2);
      scale |= static_cast<unsigned>(bytes[row * nb + k / kMxBlock]) << (8 * u);
    }
    if (4 * q + u < ks)
      *reinterpret_cast<unsigned*>(codes + (grp * ks + 4 * q + u) * kUnitBytes + r * kUnitK + 4 * c) = v;
  }
  if ((c & 3) == 0) scales[(grp * quads + q) * 64 + 16 * (c >> 2) + r] = scale;
}

hipError_t launch_mx_tile(const uint8_t* packed, const uint8_t* bytes, int K, int N, uint8_t* codes,
                          uint32_t* scales, hipStream_t s) {
  hipLaunchKernelGGL(k_mx_tile, dim3(static_cast<unsigned>(N / 16) * mx_quads(K)), dim3(256), 0, s, packed, bytes,
                     K, codes, scales);
  return hipGetLastError();
}

// Tiled codes and scales -> rows of values; same lane mapping as k_mx_quantize. Every value
// of the format is exact in bf16 and fp32 down to their subnormals; in fp16, values past
// its range round to an infinity and values below its subnormals round to them or to zero.
template <int TYPE>
__global__ __launch_bounds__(256) void k_mx_dequantize(MxDequantArgs a) {
  const int lane = threadIdx.x & 63, r = 4 * (threadIdx.x >> 6) + (lane >> 4), c = lane & 15;
  const int quads = mx_quads(a.K), ks = mx_ks(a.K);
  const int64_t grp = blockIdx.x / quads;
  const int q = blockIdx.x - static_cast<int>(grp) * quads;
  const int64_t row = grp * 16 + r;
  if (row >= a.M) return;
  unsigned v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    v[u] = 4 * q + u < ks ? *reinterpret_cast<const unsigned*>(a.codes + (grp * ks + 4 * q + u) * kUnitBytes +
                                                               r * kUnitK + 4 * c)
                          : 0u;
  const unsigned scale = a.scales[(grp * quads + q) * 64 + 16 * (c >> 2) + r];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int k = 512 * q + 128 * u + 8 * c;
    if (k >= a.K) continue;
    const float s = mx_scale_operand((scale >> (8 * u)) & 255u);
    if constexpr (TYPE == kMxF32) {
      float* dst = static_cast<float*>(a.out) + row * a.ldo + k;
      const v2f p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], s, 0);
      const v2f p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], s, 1);
      const v2f p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], s, 2);
      const v2f p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v[u], s, 3);
      *reinterpret_cast<v4f*>(dst) = v4f{p0[0], p0[1], p1[0], p1[1]};
      *reinterpret_cast<v4f*>(dst + 4) = v4f{p2[0], p2[1], p3[0], p3[1]};
    } else {
      typedef typename std::conditional<TYPE == kMxF16, F16, B16>::type T;
      *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + row * a.ldo + k) = mx_values8<T>(v[u], s);
    }
  }
}

hipError_t launch_mx_dequantize(const MxDequantArgs& a, int type, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.M + 15) / 16) * mx_quads(a.K));
  if (type == kMxF16) hipLaunchKernelGGL(k_mx_dequantize<kMxF16>, grid, dim3(256), 0, s, a);
  else if (type == kMxBf16) hipLaunchKernelGGL(k_mx_dequantize<kMxBf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_mx_dequantize<kMxF32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace i8mm
