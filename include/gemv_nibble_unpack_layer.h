/*
 * gemv_nibble_unpack_layer.h -- C ABI of the operators between a decoder
 * layer's low-bit products (MI355X, gfx950): the residual norm whose output is
 * the 8-bit rows that the products read, the append of new keys and values to
 * a paged 8-bit cache with the position rotation on the way, and attention
 * over that cache. Same library, status codes and conventions as
 * gemv_nibble_unpack.h (device pointers, caller-owned buffers, asynchronous on
 * `stream`, nothing allocated, nothing synchronised, every argument checked
 * before a launch); what differs is said here.
 *
 * The 8-bit KV cache
 * ------------------
 * A pool of num_pages pages of page_size tokens (16, 32, 64 or 128):
 *   k_codes  [num_pages, kv_heads, page_size, DP]   one byte per element
 *   v_codes  [num_pages, kv_heads, DP, page_size]   (values transposed: the
 *            attention kernel's matrix operand reads 16 tokens of a dim)
 *   k_scale, v_scale  float32 [num_pages, kv_heads]: one scale for each page
 *            of tokens and head, not negative; an element is code * scale.
 * DP is kv8_padded_dim(head_dim): head_dim rounded up to 64, 96, 128, 192 or
 * 256; the codes of dims past head_dim are zero (allocate the pool zeroed,
 * rope_append_kv8 writes zeros there). Codes are INT8 in [-127, 127] (W4_Q_I8)
 * or OCP FP8 E4M3 (W4_Q_F8); the key and the value pool have the same kind.
 * Token p of sequence b lies in slot p % page_size of page
 * page_table[b, p / page_size]; page_table is int32 [batch, table_cols], and
 * entries past a sequence's last page are never read.
 *
 * Ragged batches: sequence b's new tokens are rows q_indptr[b] ..
 * q_indptr[b+1]-1 of the token-major inputs (q_indptr int32 [batch+1], device);
 * q_indptr NULL means one new token per sequence (row b). kv_len[b] (int32,
 * device) counts the sequence's tokens INCLUDING the new ones, for both calls:
 * new token i of n has position kv_len[b] - n + i. max_q is a host bound on
 * the new tokens of any sequence. Sequences without new tokens are allowed.
 */
#ifndef GEMV_NIBBLE_UNPACK_LAYER_H
#define GEMV_NIBBLE_UNPACK_LAYER_H

#include "gemv_nibble_unpack.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit code kinds */
#define W4_Q_I8 0   /* INT8 in [-127, 127]                                      */
#define W4_Q_F8 1   /* OCP FP8 E4M3 (largest magnitude 448)                     */
/* rotary pair layouts */
#define W4_ROPE_HALF        0  /* dim i turns with dim i + rot/2                */
#define W4_ROPE_INTERLEAVED 1  /* dim 2i turns with dim 2i + 1                  */

#define W4_MAX_HEAD_DIM 256

/*
 * add_rmsnorm_q8 -- residual addition, root-mean-square norm and per-row 8-bit
 * codes in one pass over the rows:
 *   h = x + residual (float32; residual NULL: h = x),
 *   residual_out = h rounded to the input type (NULL to skip; may be X or
 *   residual itself),
 *   y = h / sqrt(mean_k(h^2) + eps) * weight (float32, not stored),
 *   y_scale[m] = max_k |y| / 127 (W4_Q_I8) or / 448 (W4_Q_F8),
 *   Yq = rint(y / y_scale) or E4M3(y / y_scale), both half-to-even; a row of
 *   zeros gets scale 0 and codes 0. A row that holds a NaN or an infinity gets
 *   scale NaN and codes 0.
 * The codes and scales are what w4a8_gemm, w2a8_gemm, w8a8_gemm (W4_Q_I8) and
 * f8f8_gemm (W4_Q_F8) take as Aq and a_scale. Everything is computed in
 * float32; y / y_scale is evaluated as (h * weight) * (127 / max|h * weight|),
 * where the root cancels, so a code can differ from the formula's by one where
 * the quotient lies within float32 rounding of a tie.
 * Float32 rows of any magnitude keep a whole scale (the squares' sum is taken
 * again with a factor where it leaves float32's range, or falls below 2^-100
 * beside a smaller eps); the products h * weight have float32's range: one that
 * overflows counts as an infinity.
 *   X, residual, residual_out [M,K], weight [K]: fp16 or float32 per in_dtype
 *   (W4_IN_F16, W4_IN_F32), 16-byte aligned. Yq 1 byte x [M,K], 16-byte
 *   aligned; y_scale float32 [M]. K a multiple of 8, at most W4_MAX_K; M >= 0
 *   (M = 0 returns W4_OK without a launch); eps >= 0 and finite.
 * Errors: W4_ERR_NULL, W4_ERR_ARG (in_dtype, q_dtype, eps), W4_ERR_SHAPE,
 * W4_ERR_ALIGN, W4_ERR_HIP.
 */
int add_rmsnorm_q8(const void* X, const void* residual, const void* weight, int in_dtype, int M,
                   int K, float eps, int q_dtype, void* residual_out, void* Yq, float* y_scale,
                   hipStream_t stream);

/* The padded head dim of a cache (64, 96, 128, 192 or 256), or 0 if head_dim is
 * not a multiple of 4 in [4, W4_MAX_HEAD_DIM]. */
int kv8_padded_dim(int head_dim);

/*
 * rope_append_kv8 -- rotate the new queries and keys by their positions, code
 * the new keys and values to 8 bits and write them into the cache.
 *   q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim]: fp16 or
 *   float32 per in_dtype; a token's heads are dense, tokens are q_stride,
 *   k_stride, v_stride elements apart (slices of a fused projection's rows
 *   need no copy). q NULL: keys and values only. q_out fp16 [tokens, q_heads,
 *   head_dim], dense; it may be q itself when q is fp16 and dense.
 *   rope float32 [rope_rows, rot_dim]: row p holds the cosines of position p's
 *   rot_dim/2 angles, then the sines (scaled angles for long contexts, a
 *   factor on the magnitude or other bases are a matter of the table). The
 *   first rot_dim dims of a head turn (rot_dim a multiple of 4, <= head_dim;
 *   0: no rotation, rope NULL), pairs (a, b) per rope_style:
 *     a' = a cos - b sin, b' = b cos + a sin, each product and the sum rounded
 *     to float32. q_out is rounded to fp16 once.
 *   Scales, for each page that gets new tokens, each head, K and V apart:
 *     m = the largest magnitude among the new elements;
 *     W4_Q_I8: s = m / 127; W4_Q_F8: s = 2^ceil(log2(m / 448)) (m / 448 in
 *     float32; at least 2^-126), so that re-coding by a ratio of two scales
 *     is exact short of subnormal codes;
 *     a page begun by this call (its slot 0 is new) takes s, and its slots past
 *     the new tokens are cleared; another page takes max(s, old scale), its
 *     earlier slots are re-coded by old scale / new scale (float32 ratio and
 *     product, then rounded to a code) where that is not 1, and its later
 *     slots are left alone. code = rint(x / s) or E4M3(x / s); s = 0 gives
 *     codes 0. A NaN or infinity among the new elements makes the page's scale
 *     of that head NaN (its codes stay finite; the page is whole again once it
 *     is begun anew).
 *   A page that gets new tokens must belong to one sequence only.
 * A sequence whose lengths do not fit (more than max_q new tokens, kv_len below
 * its new tokens, past table_cols * page_size or past rope_rows, q_indptr
 * decreasing or outside [0, tokens]) is skipped whole; a page number outside
 * [0, num_pages) skips that page's keys and values. Nothing is read or
 * written out of bounds.
 *   Alignment: q, k, v, q_out 8 bytes (fp16) or 16 bytes (float32), strides
 *   multiples of 4, codes 16 bytes, rope 16 bytes, the rest natural.
 *   q_heads a multiple of kv_heads; batch = 0, tokens = 0 or max_q = 0 return
 *   W4_OK without a launch. Errors as above, W4_ERR_ARG for an unknown
 *   in_dtype, q_dtype or rope_style.
 */
int rope_append_kv8(const void* q, const void* k, const void* v, int in_dtype, int64_t q_stride,
                    int64_t k_stride, int64_t v_stride, const float* rope, int rope_rows,
                    int rot_dim, int rope_style, const int32_t* q_indptr, const int32_t* kv_len,
                    const int32_t* page_table, int batch, int tokens, int max_q, int table_cols,
                    int q_heads, int kv_heads, int head_dim, int page_size, int num_pages,
                    int q_dtype, void* k_codes, void* v_codes, float* k_scale, float* v_scale,
                    uint16_t* q_out, hipStream_t stream);

/*
 * paged_attn_kv8_workspace_bytes -- device workspace a paged_attn_kv8 call
 * with these sizes needs (0 if none or if an argument is invalid; never more
 * than W4_ATTN_WORKSPACE_MAX). The same zero-fill and sharing rules as
 * w4_workspace_bytes, so one buffer serves matmuls and attention of a stream.
 */
#define W4_ATTN_WORKSPACE_MAX (64 * 1024 * 1024)
size_t paged_attn_kv8_workspace_bytes(int batch, int tokens, int max_q, int max_kv, int q_heads,
                                      int kv_heads, int head_dim);

/*
 * paged_attn_kv8 -- causal attention of the new tokens over the cache (after
 * rope_append_kv8): for new token i (position p), head h, kv head h' =
 * h / (q_heads / kv_heads):
 *   s_j = sm_scale * sum_d q[d] * k[j,d] for j = 0 .. p,  w = softmax(s),
 *   out = sum_j w_j * v[j]  (fp16), lse = ln sum_j exp(s_j) (float32, natural
 *   log; NULL to skip).
 * Scores, softmax statistics and sums are float32; the codes enter the matrix
 * cores as exact fp16 values, the weights w are rounded to fp16 for the second
 * product (their relative error 2^-11, as the fp16 output's). They are rounded
 * together with the value scales, in units of the largest one, r, that the row's
 * block has met: where w_j * v_scale_j is below 2^-20 of the largest w times r,
 * the error is up to 2^-31 of that product instead (the values of pages whose
 * scales lie that far apart). A token
 * that sees nothing (kv_len too small) gets out 0 and lse -inf. Codes past a
 * sequence's length are never used, whatever they hold.
 *   q fp16 [tokens, q_heads, head_dim], tokens q_stride elements apart, heads
 *   dense, 8-byte aligned, q_stride a multiple of 4; out fp16 dense [tokens,
 *   q_heads, head_dim], 8-byte aligned; lse float32 [tokens, q_heads]. max_kv
 *   is a host bound on kv_len (the launch is sized by it; a much larger bound
 *   only costs blocks that exit at once), at most 2^30. A sequence whose lengths
 *   do not fit (more than max_q new tokens: its first max_q; kv_len negative,
 *   above max_kv or past table_cols * page_size) and rows that see a token on a
 *   page number outside [0, num_pages) get NaN; a sequence whose q_indptr is
 *   decreasing or outside [0, tokens] is skipped (if that lets other sequences
 *   share rows or take them out of order, their outputs are unspecified, and
 *   still nothing is read or written out of bounds).
 * Errors as rope_append_kv8 (W4_ERR_ARG also for a sm_scale that is not
 * finite), plus W4_ERR_WORKSPACE.
 */
int paged_attn_kv8(const uint16_t* q, int64_t q_stride, const void* k_codes, const void* v_codes,
                   const float* k_scale, const float* v_scale, const int32_t* q_indptr,
                   const int32_t* kv_len, const int32_t* page_table, int batch, int tokens,
                   int max_q, int max_kv, int table_cols, int q_heads, int kv_heads, int head_dim,
                   int page_size, int num_pages, int q_dtype, float sm_scale, uint16_t* out,
                   float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_NIBBLE_UNPACK_LAYER_H */
