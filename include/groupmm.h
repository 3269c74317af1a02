/*
 * groupmm.h - C ABI of libint8mm.so, continued: products whose rows have weights of their
 * own, on MI355X (gfx950). A mixture-of-experts layer for many tokens (routing,
 * products grouped by expert, the weighted sum back to tokens), and low-rank adapters of
 * many requests beside a shared projection. The limits are those of mx4mm.h: at most
 * 2^24 rows of any operand but moe_combine's P.
 *
 * Conventions are those of int8mm.h and mx4mm.h: device pointers owned by the caller, no
 * overlap unless a call says so; matrices, weights and workspaces 16-byte aligned, vectors of
 * int32 and fp32 (offsets, rows, slots, ids, weights, scales, ranks) by their element;
 * nothing is allocated or kept; calls are asynchronous on `stream` and can be captured into a
 * HIP graph; argument errors are found on the host before any HIP call and returned as
 * int8mm_status codes. Calls that may run at the same time need workspaces of their own,
 * whose contents do not matter. The same inputs give the same bits.
 * What is in device memory is not looked at by the host: an index that is out of range is
 * taken as each call says and never reaches memory outside the operands.
 */
#ifndef GROUPMM_H_
#define GROUPMM_H_

#include "mx4mm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Routing of T tokens. p = softmax(logits[t]); the top_k largest are chosen (ties: lowest
 * expert first) with their p, divided by the sum of the chosen ones' if renormalize is not 0;
 * an expert at -inf is off, and a NaN counts as the largest logit, as in moe_layer.
 *   logits        [T, E] contiguous, logits_dtype any mx4_dtype; 1 <= T <= 2^24, 1 <= E <= 512,
 *                 1 <= top_k <= min(E, 16).
 *   ids, weights  out, int32 and fp32 [T, top_k], in descending order (id -1 and weight 0 past
 *                 the last expert that is on).
 *   offsets       out, int32 [E + 1]: expert e has rows offsets[e] up to offsets[e + 1] of a
 *                 product grouped by expert, its tokens in ascending order.
 *   rows          out, int32 [T top_k]: the token of each of those rows, -1 behind the last.
 *   slots         out, int32 [T, top_k]: the row of each pair of token and place, -1 for none.
 *   workspace     at least moe_route_workspace_bytes(T, E) bytes (0 up to 64 tokens, then it
 *                 may be NULL, and on bad shapes).
 * One launch up to 64 tokens, two beyond.
 */
size_t moe_route_workspace_bytes(int64_t T, int64_t E);
int moe_route(const void* logits, int64_t T, int64_t E, int logits_dtype, int64_t top_k, int renormalize,
              int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace,
              size_t workspace_bytes, hipStream_t stream);

/*
 * Products grouped by expert: row p of Y, offsets[e] <= p < offsets[e + 1], is the product of
 * row rows[p] of X with expert e's N rows of the weight.
 *   weight_format 0: int8, as int8_mixed_matmul (the outlier columns are those of the whole of
 *                 X; more than max_outliers of them fill the experts' rows with NaN); X is fp16
 *                 and contiguous.
 *                 1: MX4, as mx4_matmul (X is quantized in the call); threshold and
 *                 max_outliers are not looked at.
 *   X             [M, K], row stride ldx, dtype MX4_F16 or MX4_BF16; M and P at most 2^24; less
 *                 than 2^33 elements of X and of one expert's weight with MX4 weights.
 *   w, s          one prepared weight of E * N output features over K.
 *   offsets       int32 [E + 1], ascending from 0; 1 <= E <= 1024. Offsets that do not ascend,
 *                 or lie outside 0 .. P, give rows of Y that mean nothing.
 *   rows          int32 [P], or NULL: row p of X, and P = M. A row outside 0 .. M - 1 counts as
 *                 zeros.
 *   gated         0: Y is [P, N]. Otherwise an expert's N features are N / 2 gate features and
 *                 then as many up features (N a multiple of 32), and Y [P, N / 2] is
 *                 silu(gate) * up, rounded once.
 *   Y             out, contiguous, dtype. Rows behind offsets[E] are zeros.
 *   workspace     at least moe_grouped_workspace_bytes(...) bytes (0 on bad shapes).
 */
size_t moe_grouped_workspace_bytes(int64_t M, int64_t K, int64_t P, int64_t E, int64_t N, int weight_format,
                                   int64_t max_outliers);
int moe_grouped_matmul(const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, int weight_format, const void* w,
                       const void* s, int64_t E, int64_t N, const int32_t* offsets, const int32_t* rows, int64_t P,
                       int gated, float threshold, int64_t max_outliers, void* Y, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

/*
 * Y[t] = sum over j of weights[t, j] P[slots[t, j]], summed in fp32 in the order of j, rounded
 * once; a slot outside 0 .. P_rows - 1 adds nothing.
 *   P             [P_rows, D] contiguous, dtype MX4_F16 or MX4_BF16; D a multiple of 16.
 *   slots, weights  int32 and fp32 [T, top_k], 1 <= T <= 2^24, 1 <= top_k <= 16; P_rows up to 2^28.
 *   Y             out, [T, D] contiguous, dtype.
 */
int moe_combine(const void* P, int64_t P_rows, int64_t D, int dtype, const int32_t* slots, const float* weights,
                int64_t T, int64_t top_k, void* Y, hipStream_t stream);

/*
 * Low-rank adapters beside a shared projection: with a = ids[m],
 *   out[m] = Y[m] + scales[a] B_a (A_a X[m]),
 * fp32 sums, one rounding. The sums A X enter the second product whole in bf16, and in fp16 within
 * 2^-23 of each or 2^-39 of their row's largest, whichever is more. Rows whose id is outside
 * 0 .. S - 1 have no adapter and keep Y[m]. An infinity or a NaN in a row of X, or in what an
 * adapter's ranks hold, gives NaNs wherever it enters, also against zeros.
 *   Y, X, out     [M, N], [M, K], [M, N], row strides ldy, ldx, ldo, dtype MX4_F16 or MX4_BF16.
 *                 out may be Y (then ldo = ldy): the adapters are added in place.
 *   A, B          [S, R, K] and [S, N, R] contiguous, dtype; 1 <= S <= 1024, R a multiple of 8,
 *                 8 <= R <= 128.
 *   ids           int32 [M], in any order.
 *   scales        fp32 [S], or NULL: 1.
 *   ranks         int32 [S], or NULL: R. Adapter a has min(ranks[a], R) ranks, and what A and B
 *                 hold beyond them is not looked at.
 *   workspace     at least lora_workspace_bytes(M, K, S, R) bytes (0 on bad shapes).
 * Up to 64 rows are two launches, more three.
 */
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t S, int64_t R);
int lora_apply(const void* Y, int64_t ldy, const void* X, int64_t M, int64_t K, int64_t ldx, int dtype, const void* A,
               const void* B, int64_t S, int64_t R, int64_t N, const int32_t* ids, const float* scales,
               const int32_t* ranks, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
               hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GROUPMM_H_ */
