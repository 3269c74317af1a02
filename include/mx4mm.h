/*
 * mx4mm.h - C ABI of libint8mm.so, continued: products with microscaled 4-bit ("MX4")
 * operands, and a mixture-of-experts layer for a few tokens over int8 or MX4 weights,
 * on MI355X (gfx950).
 *
 * MX4: a row of K elements is cut into blocks of 32 consecutive ones (the last may hold
 * 16). A block holds one power of two 2^s with s = clamp(floor(log2 max|x|) - 2, -127,
 * 127), stored as the byte s + 127, and a 4-bit code of each x / 2^s: bit 3 the sign,
 * bits 0-2 an index into {0, 0.5, 1, 1.5, 2, 3, 4, 6}, to the nearest, ties to the even
 * index, anything beyond 6 to 6. A block of zeros has byte 0. A block with an infinity or
 * a NaN has byte 255 and codes 0, and all its elements read back as NaN: unlike the int8
 * calls, these take inputs that are not finite, and a product's output is NaN where the
 * row or the column holds such a block.
 *
 * The tiled layout, for activations (rows = tokens) and weights (rows = output features)
 * alike, of R rows (padded to 16) and K elements, KS = ceil(K / 128), Q = ceil(KS / 4):
 *   codes   element (r, k) is in byte
 *             ((r / 16) * KS + k / 128) * 1024 + (r % 16) * 64 + (k % 128) / 2,
 *           even k in the low four bits; mx4_codes_bytes(R, K) bytes.
 *   scales  the byte of block (r, b = k / 32) is byte
 *             ((r / 16) * Q + b / 16) * 256 + ((b % 4) * 16 + r % 16) * 4 + (b / 4) % 4;
 *           mx4_scales_bytes(R, K) bytes.
 * All padding is codes 0 and byte 0.
 *
 * Conventions are those of int8mm.h: device pointers, 16-byte aligned, owned by the
 * caller, no overlap; nothing is allocated or kept; calls are asynchronous on `stream` and
 * can be captured into a HIP graph; argument errors are found on the host before any HIP
 * call and returned as int8mm_status codes (int8mm_strerror). K and N are multiples of 16,
 * 16 <= K <= 2^20, 16 <= N <= 2^24, 1 <= M <= 2^24, and no operand has more than 2^36
 * elements. `dtype` is an mx4_dtype; a value that a call does not take is
 * INT8MM_E_SHAPE. Row strides (ldx, ldo) are in elements, multiples of 8 and at least K.
 */
#ifndef MX4MM_H_
#define MX4MM_H_

#include "int8mm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx4_dtype { MX4_F16 = 0, MX4_BF16 = 1, MX4_F32 = 2 } mx4_dtype;

/* Bytes of the tiled codes and scales of `rows` rows of K elements (0 on bad shapes). */
size_t mx4_codes_bytes(int64_t rows, int64_t K);
size_t mx4_scales_bytes(int64_t rows, int64_t K);

/* Rows of X [M, K] (row stride ldx; MX4_F16 or MX4_BF16) to MX4. */
int mx4_quantize(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, uint8_t* codes,
                 uint8_t* scales, hipStream_t stream);

/*
 * A weight to MX4, once at load: rows are the N output features. w_layout 0: W [K, N]
 * row-major; 1: W [N, K] row-major (then the same as mx4_quantize). Contiguous.
 */
int mx4_prepare_weight(const void* W, int64_t K, int64_t N, int w_layout, int dtype,
                       uint8_t* codes, uint8_t* scales, hipStream_t stream);

/*
 * An MX4 weight that a checkpoint holds row by row to the tiled layout, no arithmetic:
 *   packed       uint8 [N][16 ceil(K / 32)]: element 2 i of a row in the low four bits of
 *                its byte i; codes past K are ignored.
 *   block_scales uint8 [N][ceil(K / 32)].
 */
int mx4_tile_weight(const uint8_t* packed, const uint8_t* block_scales, int64_t K, int64_t N,
                    uint8_t* codes, uint8_t* scales, hipStream_t stream);

/*
 * The values of tiled codes and scales: out [M, K], row stride ldo, any mx4_dtype. Exact in
 * MX4_F32 and MX4_BF16, but values of 2^128 and more, which only a weight from mx4_tile_weight
 * can hold (bytes 253 and 254), become infinities, there and where a product takes the
 * weight's values as bf16; in MX4_F16 rounded once where the value is outside fp16's range.
 */
int mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, int dtype,
                   void* out, int64_t ldo, hipStream_t stream);

/*
 * Y [M, N] = MX4(X) W^T: X is quantized as by mx4_quantize, the products of codes are scaled
 * by both blocks' powers of two and accumulated in fp32, Y is rounded once to dtype
 * (MX4_F16 or MX4_BF16, X's type).
 * Few rows (M <= 16, and up to 64 with M ceil(K / 512) <= 96) are one launch, without a
 * workspace, and need M ldx < 2^30; more are a quantization launch and the product (M <= 64
 * a weight stream, beyond that output tiles; where K is long and the tiles are few, K is
 * split and a third launch joins the sums).
 *   workspace   at least mx4_matmul_workspace_bytes(M, K, N) bytes (0 for the few rows above,
 *               then workspace may be NULL, and on bad shapes); its contents do not matter.
 *               Calls that may run at the same time need workspaces of their own.
 */
size_t mx4_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N);
int mx4_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype,
               const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, void* Y,
               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The product alone, X already MX4 (mx4_quantize): once for several weights.
 *   workspace   at least mx4_matmul_q_workspace_bytes(M, K, N) bytes; often 0 (and on bad
 *               shapes), then workspace may be NULL. Otherwise as for mx4_matmul.
 */
size_t mx4_matmul_q_workspace_bytes(int64_t M, int64_t K, int64_t N);
int mx4_matmul_q(const uint8_t* x_codes, const uint8_t* x_scales, int64_t M, int64_t K,
                 const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, int dtype, void* Y,
                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Y [M, N] = X W^T with X as it is, for a few tokens: 1 <= M <= 16 and M ldx < 2^30 (X is
 * read through a buffer resource). fp32 accumulation, one rounding to dtype (MX4_F16 or
 * MX4_BF16). The weight values enter exactly, however far apart a row's blocks are; but with
 * fp16 X those of a block of byte 0 (below 2^-124) may count as zeros beside larger ones. A
 * row of X with an infinity or a NaN gives infinities or NaNs.
 */
int mx4_weight_only_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype,
                           const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, void* Y,
                           hipStream_t stream);

/*
 * A mixture-of-experts layer for T <= 16 tokens, from router logits to the output, with
 * weights held in int8 or MX4 and 16-bit activations:
 *   p = softmax(logits[t]), the top_k largest chosen (ties: lowest expert first), their p
 *       divided by the sum of the chosen ones' if renormalize is not 0;
 *   Y[t] = sum over the chosen e of p_e Down_e (silu(Gate_e X[t]) * (Up_e X[t])).
 * An expert whose logit is -inf is off for the token; where fewer than top_k are on, the
 * rest of the list is empty, and a token with none (a padding row) gets zeros and costs no
 * weight traffic. A NaN counts as the largest logit and makes the token's output NaN, and so
 * does a logit of +inf.
 *   X             [T, D], row stride ldx (a multiple of 8, >= D, T ldx < 2^30), dtype
 *                 MX4_F16 or MX4_BF16.
 *   logits        [T, E] contiguous, logits_dtype any mx4_dtype; 1 <= E <= 512,
 *                 1 <= top_k <= min(E, 16).
 *   weight_format 0: int8 (w13, w2 unit-tiled, s13, s2 their fp32 column constants, as from
 *                 int8_prepare_weight / int8_tile_weight), 1: MX4 (tiled codes and scales).
 *   w13, s13      one prepared weight of E * 2 I output features over K = D: for each
 *                 expert its I gate rows, then its I up rows.
 *   w2, s2        one prepared weight of E * D output features over K = I.
 *                 D and I are multiples of 16, at most 2^20 (int8: 133144).
 *   Y             out, [T, D] contiguous, dtype.
 *   ids, weights  out, nullable: int32 and fp32 [T, top_k], the lists in descending order
 *                 (id -1 and weight 0 past the last chosen expert).
 *                 One expert's row groups are a prepared weight by themselves (2 I and D are
 *                 multiples of 16): more than 16 tokens go through here 16 at a time, or, a
 *                 prompt's, through the products (mx4_matmul, int8_mixed_matmul) expert by
 *                 expert on the rows of X that chose it.
 *   workspace     at least moe_layer_workspace_bytes(T, I, top_k) bytes; its contents do not
 *                 matter. Calls that may run at the same time need workspaces of their own.
 * fp32 sums and hidden values, weight values as in mx4_weight_only_matmul; one rounding of Y.
 * The same inputs give the same bits.
 */
size_t moe_layer_workspace_bytes(int64_t T, int64_t I, int64_t top_k);
int moe_layer(const void* X, int64_t T, int64_t D, int64_t ldx, int dtype, const void* logits,
              int64_t E, int logits_dtype, int64_t top_k, int renormalize, int weight_format,
              const void* w13, const void* s13, const void* w2, const void* s2, int64_t I,
              void* Y, int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
              hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MX4MM_H_ */
