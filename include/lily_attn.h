/*
 * lily_attn.h -- C ABI of the attention side of a decoder block, next to the
 * MoE expert layer of lily_moe.h (same library, conventions, error codes and
 * status word).
 *
 * The model of the pages keeps 16 query heads over 2 key/value heads in its
 * attention layers (page "Lily Beats MLX-LM 1.35x on Decode: Perplexity's
 * Rust+Metal Engine for Apple Silicon", section "Model structure and three
 * workload shapes").  The operators, in the order a block uses them:
 *   lily_attn_add_rmsnorm    residual += x; RMSNorm of the sum, as bf16/fp16
 *                            rows (what lily_moe_* takes) or 8-bit rows with
 *                            scales (what 8-bit projections take)
 *   lily_attn_rope_append    rotate q and k by position, append k and v to a
 *                            paged cache
 *   lily_attn_shared_prefix  attention of a batch whose sequences share a
 *                            prefix (a system prompt, a document) and go on
 *                            in pages of their own
 * and, for a cache of 8-bit codes with a scale for each token and head,
 *   lily_attn_rope_append8   the same as lily_attn_rope_append into codes
 *   lily_attn_decode8        attention of new tokens over it
 *
 * Conventions are lily_moe.h's: device pointers, 16-byte aligned (arrays of
 * indices, lengths, frequencies and lse: by their elements), caller-owned;
 * nothing is allocated or synchronised; every launch goes to `stream`; on an
 * argument error nothing is launched.  The workspace of both appends and of
 * attention is zero-filled once before its first use and starts with a
 * status word that lily_moe_status() reads and clears.
 */
#ifndef LILY_ATTN_H
#define LILY_ATTN_H

#include "lily_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types beside LILY_DTYPE_BF16 and LILY_DTYPE_F32. */
#define LILY_DTYPE_F16 2
#define LILY_DTYPE_E4M3 3 /* 4-bit exponent, 3-bit mantissa, largest value 448 */

/* Device status bits beside lily_moe.h's. */
#define LILY_STATUS_BAD_PAGE 0x10u /* a page index outside the cache: its keys were skipped   */
#define LILY_STATUS_BAD_SLOT 0x20u /* an append slot outside the cache: the token was skipped */
#define LILY_STATUS_BAD_LEN 0x40u  /* a sequence length or token range outside its bounds: it
                                      was clamped                                             */

/* ------------------------------------------------------------ add + RMSNorm
 * T, d          rows and row width; T >= 1, 1 <= d <= 16384
 * x_dtype       BF16, F16 or F32
 * res_dtype     BF16, F16 or F32: type of residual and residual_out
 * w_dtype       BF16, F16 or F32
 * out_dtype     BF16, F16 or E4M3
 * group         columns that share a scale (E4M3): 0 = the whole row, else 64
 *               or 128 and a divisor of d; 0 for BF16 and F16
 * eps           added to the mean square
 * *_stride      elements from one row to the next (>= d)
 */
typedef struct {
  int32_t T, d, x_dtype, res_dtype, w_dtype, out_dtype, group;
  float eps;
  int64_t x_stride, res_stride, res_out_stride, out_stride;
} lily_attn_norm_dims;

/* r = residual + x (fp32), n = r / sqrt(mean(r^2) + eps) * weight, and
 *   residual_out = r rounded to res_dtype,
 *   out = n rounded to BF16 / F16; or, E4M3, out = n / s rounded with
 *   s = max|n| / 448 over each group of columns (0 where that is 0 or rounds to
 *   0, and out is 0).
 * The norm is taken of the fp32 sum, before the residual's rounding.  The 8-bit
 * code is that of n times 448 / max|n|, a reciprocal rounded to fp32, or of n / s
 * in rows read element by element: next to a border between two codes either may
 * come out, and rows of another alignment may differ in such a code.
 *   residual      NULL: r = x
 *   weight        [d], or NULL: ones
 *   residual_out  may be residual itself (in place), or NULL: not stored
 *   scales        fp32 [T][d / group] ([T] when group is 0): E4M3 only, else NULL
 * Rows that all lie on multiples of eight elements are read and written in
 * vectors, and so are, without groups, rows of odd widths whose operands have the
 * same distance from one (as contiguous tensors do); others element by element.
 * A row with a NaN or an infinity gives NaN there
 * (E4M3: its scale too). */
int lily_attn_add_rmsnorm(const lily_attn_norm_dims* dims, const void* x, const void* residual,
                          const void* weight, void* residual_out, void* out, float* scales,
                          void* stream);

/* -------------------------------------------------------------- paged cache
 * K and V live in n_pages pages of page_size tokens; the element (page, head,
 * token in page, i) of either is at page*page_stride + head*head_stride +
 * token*token_stride + i.  Both [page][token][head][D] and [page][head][token][D]
 * are described so, and so is a K and V pair interleaved in one allocation.
 * Pages a call names hold its tokens; other contents are never used, whatever
 * their bits.
 *   dtype       BF16 or F16
 *   page_size   16, 32, 64, 128 or 256
 *   n_kv_heads  1 to 256
 *   head_dim    a multiple of 8, 8 to 256
 *   strides     multiples of 8 elements, below 2^39
 */
typedef struct {
  void* k;
  void* v;
  int32_t dtype, n_pages, page_size, n_kv_heads, head_dim;
  int64_t page_stride, head_stride, token_stride;
} lily_attn_cache;

/* ------------------------------------------------------------- RoPE, append
 * T            tokens
 * n_q_heads    query heads (any number)
 * rotary_dim   leading dimensions of a head that rotate: even, 0 to head_dim
 * style        0: pairs (i, i + rotary_dim/2); 1: pairs (2i, 2i + 1)
 * strides      elements, per token and per head, of q, k, v and q_out:
 *              multiples of 8, below 2^31
 */
typedef struct {
  int32_t T, n_q_heads, rotary_dim, style;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
  int64_t v_token_stride, v_head_stride, qo_token_stride, qo_head_stride;
} lily_attn_rope_dims;

/* The pair (a, b) number i of token t turns by the angle positions[t] *
 * inv_freq[i]: (a cos - b sin, b cos + a sin), in fp32, rounded once.  The
 * frequency is taken as a 64-bit fraction of a turn, cut off, and the product with
 * the position keeps its last 64 bits: the angle is off by less than position *
 * 2^-64 of a turn (2^-33 at 31 bits), which its rounding to fp32 for the sines
 * (2^-26 of a turn) hides.
 *   positions   int32 [T]
 *   inv_freq    fp64 [rotary_dim / 2], radians per position
 *   slots       int64 [T]: token t goes to page slots[t] / page_size, row
 *               slots[t] % page_size; negative: the token is not appended; at or
 *               past n_pages*page_size: LILY_STATUS_BAD_SLOT, not appended.  Two
 *               tokens with one slot leave either's values there.
 *   q           [T][n_q_heads][D], written rotated to q_out (may be q itself);
 *               NULL (and q_out NULL, n_q_heads 0): append only
 *   k, v        [T][n_kv_heads][D]; both NULL: rotate q only (slots then unused)
 *   workspace   at least 256 bytes (the status word) */
int lily_attn_rope_append(const lily_attn_rope_dims* dims, const lily_attn_cache* cache,
                          const void* q, const void* k, const void* v, const int32_t* positions,
                          const int64_t* slots, const double* inv_freq, void* q_out,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------- attention with a shared prefix
 * n_tokens     query rows of the batch, 1 to 65536
 * n_q_heads    a multiple of the cache's n_kv_heads, at most 64 per KV head
 * n_seqs       sequences, 1 to 65536
 * max_q_len    at least every sequence's number of query tokens; 1 in decode
 * prefix_len   tokens of the shared prefix, 0 for none
 * max_seq_len  at least every sequence's own length; table_stride * page_size
 *              or less.  The launch is planned by this bound, not by the
 *              lengths, which only the device knows: the room of the sequences
 *              serves in a captured graph, a tight bound is up to a sixth faster
 * table_stride entries of block_table per sequence
 * scale        softmax scale, > 0
 * strides      elements, per token and per head, of q and out: multiples of 8
 */
typedef struct {
  int32_t n_tokens, n_q_heads, n_seqs, max_q_len, prefix_len, max_seq_len, table_stride;
  float scale;
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
} lily_attn_dims;

/* Device bytes of workspace (0 on bad dims). */
size_t lily_attn_workspace_bytes(const lily_attn_dims* dims, const lily_attn_cache* cache);

/* Which kernel a call with these dims reads the shared prefix with (host only):
 * NONE without a prefix, WARP for few rows and keys (mma.sync), TENSOR for many
 * (tcgen05).  Negative on bad dims. */
#define LILY_PREFIX_NONE 0
#define LILY_PREFIX_WARP 1
#define LILY_PREFIX_TENSOR 2
int lily_attn_prefix_kernel(const lily_attn_dims* dims, const lily_attn_cache* cache);

/* Query token j of the q_len of a sequence with seq_len own tokens (its new
 * tokens among them, appended already) sees the whole prefix and its sequence's
 * own tokens 0 .. seq_len - q_len + j.  Over those keys
 *   out = softmax(scale * q k^T) v,  lse = log(sum(exp(scale * q k^T))),
 * query heads sharing KV head h being h*G .. h*G + G-1.  A row that sees
 * nothing is 0 with lse -infinity.  The prefix is read once for all sequences.
 * Scores, softmax statistics and sums are fp32; the probabilities are rounded
 * to the cache's type for the tensor cores (fp16: scaled by 2^7 or more, so that
 * one 2^-21 times the largest still keeps all its bits).  Scores stay below 2^27
 * in size: near larger ones an fp32 number is too coarse for a softmax.
 *   q             [n_tokens][n_q_heads][D], the cache's type
 *   prefix_pages  int32 [ceil(prefix_len / page_size)]; NULL when prefix_len is 0
 *   q_start       int32 [n_seqs + 1]: sequence s owns query tokens q_start[s] ..
 *                 q_start[s + 1] - 1; NULL: max_q_len tokens each (n_tokens =
 *                 n_seqs * max_q_len).  A token of no sequence sees the prefix.
 *   seq_lens      int32 [n_seqs], own tokens (0: none)
 *   block_table   int32 [n_seqs][table_stride] page indices
 *   out           [n_tokens][n_q_heads][D], the cache's type
 *   lse           fp32 [n_tokens][n_q_heads] or NULL
 * A page index outside the cache sets LILY_STATUS_BAD_PAGE and its keys are
 * skipped; a length or range outside its bounds sets LILY_STATUS_BAD_LEN and is
 * clamped (a token that two clamped ranges share sees either's keys).  Outputs are
 * otherwise the same bits on every run with the same arguments. */
int lily_attn_shared_prefix(const lily_attn_dims* dims, const lily_attn_cache* cache,
                            const void* q, const int32_t* prefix_pages, const int32_t* q_start,
                            const int32_t* seq_lens, const int32_t* block_table, void* out,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------- 8-bit cache
 * K and V as e4m3 codes with one fp32 scale for each token and head: element i is
 * code * scale.  Codes lie in pages as lily_attn_cache's elements do; the scale of
 * (page, head, token in page) of either lies at page*scale_page_stride +
 * head*scale_head_stride + token*scale_token_stride.
 *   page_size, n_kv_heads  as lily_attn_cache's
 *   head_dim    a multiple of 16, 16 to 256
 *   strides     of codes: multiples of 16; of scales: 1 or more; below 2^39
 * k and v 16-byte aligned, scales by their elements.  A page's codes are finite
 * (as the append writes them); scales may be any finite number, or NaN, which spoils
 * the rows that see its key.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  int64_t page_stride, head_stride, token_stride;
  int64_t scale_page_stride, scale_head_stride, scale_token_stride;
} lily_attn_cache8;

/* lily_attn_rope_append into an 8-bit cache: q is rotated as there; k, rotated, and
 * v are rounded to fp32's x / s, with s = max|x| / 448 over the head, and that to
 * its code.  A head whose s is below 2^-126 becomes zeros with scale 0, one with an
 * infinity or a NaN zeros with scale NaN.
 *   dtype   BF16 or F16: type of q, k, v and q_out
 * Two tokens with one slot leave codes and a scale there that may be of either, not
 * of the same one.  Everything else is lily_attn_rope_append's. */
int lily_attn_rope_append8(const lily_attn_rope_dims* dims, const lily_attn_cache8* cache,
                           int32_t dtype, const void* q, const void* k, const void* v,
                           const int32_t* positions, const int64_t* slots, const double* inv_freq,
                           void* q_out, void* workspace, size_t workspace_bytes, void* stream);

/* Device bytes of workspace of lily_attn_decode8 (0 on bad dims). */
size_t lily_attn_decode8_workspace_bytes(const lily_attn_dims* dims, const lily_attn_cache8* cache);

/* Attention of new tokens over an 8-bit cache: query token j of the q_len of a
 * sequence with seq_len keys (its new tokens among them, appended already) sees keys
 * 0 .. seq_len - q_len + j, as in lily_attn_shared_prefix without a prefix.  Made for
 * single tokens and short runs: the keys of a KV head are read once for each 8 rows
 * (query tokens times query heads of the KV head).
 *   dims    prefix_len is 0; sequences that share pages name them in their tables
 *   dtype   BF16 or F16: type of q and out
 *   q_start, seq_lens, block_table, lse  as lily_attn_shared_prefix's
 * Scores, softmax statistics and sums are fp32, and scores stay below 2^27 in size, as
 * there; a probability times its key's value scale is rounded to fp16, held so that one
 * 2^-24 times the largest value scale, whatever that is, still keeps all its bits.  A
 * row that sees nothing is 0 with lse -infinity; tokens of no sequence are left as they
 * were.  Bad page indices, lengths and ranges are treated as by
 * lily_attn_shared_prefix, and outputs are otherwise the same bits on every run with
 * the same arguments. */
int lily_attn_decode8(const lily_attn_dims* dims, const lily_attn_cache8* cache, int32_t dtype,
                      const void* q, const int32_t* q_start, const int32_t* seq_lens,
                      const int32_t* block_table, void* out, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Give-up limit, in nanoseconds, of every wait inside shared_prefix's and decode8's
 * kernels (for a copy or another warp of the same block): 2 s by default, counted in
 * tries of some 4 us, at least one.  Returns the previous limit.  A block whose
 * wait runs out sets LILY_STATUS_TIMEOUT and ends, and that call's outputs are
 * invalid; the next call on the workspace is not affected.  For tests of the
 * error path; 0 makes the warps that compute give up at their first wait, while
 * copies are in flight.  Applies to calls issued after it. */
uint64_t lily_attn_set_wait_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif
#endif /* LILY_ATTN_H */
