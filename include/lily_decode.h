/*
 * lily_decode.h -- C ABI of what a decode step needs beside its experts
 * (lily_moe.h) and its attention (lily_attn.h): projections of a few rows by
 * 4-bit weights, up to the head's logits, and the draw of a token from them
 * (same library, conventions, error codes and status word).
 *
 * The pages stream 4-bit weights through matrix-vector products in decode and
 * put the sampled token into the next step's input slot without the host (page
 * "Lily Beats MLX-LM 1.35x on Decode: Perplexity's Rust+Metal Engine for Apple
 * Silicon", section "Decode: eliminating per-token CPU round trips").
 *
 * Conventions are lily_moe.h's: device pointers, 16-byte aligned unless it says
 * otherwise, caller-owned; nothing is allocated or synchronised; every launch goes
 * to `stream`; on an argument error nothing is launched.
 */
#ifndef LILY_DECODE_H
#define LILY_DECODE_H

#include "lily_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- 4-bit projections
 * T            rows, 1 to 32
 * K            input features, a multiple of 128, 128 to 16384
 * N            output features (any number, 1 to 2^24)
 * group        consecutive weights of a row that share a scale: 32, 64 or 128
 * x_dtype      BF16 or F16
 * out_dtype    BF16, F16 or F32
 * x_stride     elements from one row of x to the next: a multiple of 8, >= K
 * out_stride   elements from one row of y to the next: >= N
 */
typedef struct {
  int32_t T, K, N, group, x_dtype, out_dtype;
  int64_t x_stride, out_stride;
} lily_decode_linear_dims;

/* y[t][n] = sum over k of x[t][k] * (scale * q[n][k] + bias), the weights being
 * lily_moe_weights' format: codes 0..15, scale and bias of k's group.
 *   x      [T][K]
 *   q      uint8 [N][K/2]: byte j of a row holds element 2j in bits 0-3 and 2j+1
 *          in bits 4-7
 *   scale  bf16 [N][K/group]
 *   bias   bf16 [N][K/group]; NULL: -8 times the scale (symmetric weights)
 *   y      [T][N]; 16-byte aligned in its first row; shares no element with x
 * Products with the codes are exact and summed in fp32, as is everything else;
 * the sum is rounded once.  x of 2^112 or more in size overflows fp32 on the way.
 * A row of x with an infinity or a NaN gives no finite value in that row of y.
 * The result is the same bits on every run. */
int lily_decode_linear(const lily_decode_linear_dims* dims, const void* x, const uint8_t* q,
                       const uint16_t* scale, const uint16_t* bias, void* y, void* stream);

/* ------------------------------------------------------------ token sampling
 * B             rows, 1 to 65535
 * V             vocabulary, 1 to 524288
 * logits_dtype  BF16, F16 or F32
 * stride        elements from one row of logits to the next: >= V
 */
typedef struct {
  int32_t B, V, logits_dtype, reserved; /* reserved: 0 */
  int64_t stride;
} lily_decode_sample_dims;

/* One token for each row.  The row's tokens are put in order of their logits,
 * equal ones by index, the lowest first; m is the largest logit and token i has
 * the mass exp((logit[i] - m) / temperature).  Of that order are kept
 *   the first top_k tokens (top_k <= 0 or >= V: all),
 *   of these the shortest run from the first on that holds top_p of their mass
 *   or more (top_p >= 1: all; top_p <= 0: one token),
 *   of these the tokens whose mass is min_p or more (min_p <= 0: all),
 * and always the first.  The draw goes through the kept tokens in order of their
 * indices: the token is the first whose mass, added to that of those before it,
 * is above u times the mass of all that are kept.
 *   logits       [B][V]
 *   temperature  fp32 [B]; 0 or less (or NaN): the first of the order, no draw
 *   top_k        int32 [B] or NULL (all)
 *   top_p        fp32 [B] or NULL (all); NaN: all
 *   min_p        fp32 [B] or NULL (all); NaN: all
 *   u            fp32 [B], 0 <= u < 1 (held to that; NaN: 0); NULL: the first of the
 *                order in every row
 *   tokens       int32 [B]
 *   logprobs     fp32 [B] or NULL: the log of the token's share of the kept mass; 0 in
 *                rows without a draw (temperature 0 or less, or u NULL)
 *   workspace    256 bytes or more (the status word, as lily_attn.h's)
 * The arrays are aligned by their elements; logits by 16 bytes in their first row
 * (rows that do not lie on 16 bytes are read element by element at their ends).
 * Logits of -infinity have no mass; +infinity takes all of it (several: equal
 * shares).  A NaN counts as -infinity and sets LILY_STATUS_NAN_LOGIT.  A row of
 * nothing but these gives token -1 with logprob -infinity.
 * Masses are held as whole numbers of 2^-44 of the largest, each right to 2^-23 of
 * itself or half of such a unit, and summed without rounding: the result does not
 * depend on the order of the sums, and is the same on every run. */
int lily_decode_sample(const lily_decode_sample_dims* dims, const void* logits,
                       const float* temperature, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* u, int32_t* tokens, float* logprobs,
                       void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LILY_DECODE_H */
