/*
 * fp8lin -- the operators that a transformer on FP8-AMAX products (fp8lin.h)
 * trains with, beside those of fp8lin_block.h, in the same library
 * (libfp8lin.so):
 *   - the embedding at its start, with its gradient by sorted tokens;
 *   - norms of queries and keys for each head with the rotary positions, and
 *     their gradients (single tokens in front of the FP8 cache likewise);
 *   - attention over packed sequences, and its gradients.
 * Dtypes, status codes and the conventions for every entry point are
 * fp8lin.h's.  No output may overlap an input, another output or a workspace.
 */
#ifndef FP8LIN_TRAIN_H
#define FP8LIN_TRAIN_H

#include "fp8lin.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Embedding.  out[t] = scale * table[ids[t]], in fp32 and rounded once.
 *   ids     device, `tokens` int32 (id_bits 32) or int64 (id_bits 64).  An id
 *           outside 0 .. vocab - 1 (padding: -1) is no token: its row of out is
 *           zeros, and it has no gradient.
 *   table   device, vocab x d of table_dtype
 *   out     device, tokens x d of out_dtype, written
 * Tensors need 16-byte alignment, ids their own.  vocab, tokens >= 0, d >= 1.
 *
 * fp8_embedding_bwd: dtable[v] = scale * sum of dout[t] over the t with
 * ids[t] = v, and zeros for a v that no token has.
 *   dout       device, tokens x d of dout_dtype
 *   accumulate != 0: added to what dtable holds (one fp32 addition); rows that
 *              no token has are left as they are
 *   dtable     device, vocab x d floats, written
 *   ws         device, 16-byte aligned, fp8_embedding_bwd_workspace_bytes()
 *              bytes.  The call overwrites it and keeps no pointer; calls in
 *              flight at the same time need separate ones.
 * Tokens are sorted by id, stably, and an id's rows are added in their order
 * in fp32, in runs of at most 16 whose sums (of long runs also sums of 64 of
 * these) are added in their order: same inputs, same bits.  vocab < 2^31, tokens < 2^31 - 2^16.
 */
int fp8_embedding_fwd(const void* ids, int32_t id_bits, int64_t tokens, const void* table, fp8_dtype_t table_dtype,
                      int64_t vocab, int64_t d, float scale, void* out, fp8_dtype_t out_dtype, void* stream);
int64_t fp8_embedding_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d);
int fp8_embedding_bwd(const void* dout, fp8_dtype_t dout_dtype, const void* ids, int32_t id_bits, int64_t tokens,
                      int64_t vocab, int64_t d, float scale, int32_t accumulate, float* dtable, void* ws,
                      int64_t ws_bytes, void* stream);

/*
 * Norms of queries and keys for each head, and the rotary positions, in one
 * pass over the fused query / key / value product's rows.  For a head's x of a
 * query or key, with that side's weight w:
 *   rstd = (mean_j x_j^2 + eps)^(-1/2),  n_j = (x_j * rstd) * w_j
 *   y = n rotated by its token's position
 * in fp32, rounded to bf16 once; a value is rounded to bf16.
 *   x          device, tokens rows of q_heads + 2 kv_heads heads of head_dim (64,
 *              128 or 256) elements of x_dtype: queries, keys, values; rows
 *              x_stride elements apart
 *   wq, wk     device, head_dim values of w_dtype, or both NULL: no norm
 *   positions  device, tokens int32, or NULL: row t is at position t.  A position
 *              outside the table counts as the nearest one in it.
 *   cos, sin   device, rope_rows x head_dim / 2 floats, or both NULL: no
 *              rotation.  rope_pairs as in fp8_kv_append.  Without positions
 *              rope_rows >= tokens (FP8_ERR_SIZE).
 *   y          device, tokens x (q_heads + 2 kv_heads) x head_dim bf16 words,
 *              written
 * Row pointers and strides (in bytes) must be multiples of 16, angles and
 * weights 16-byte aligned.  q_heads, kv_heads >= 1.
 *
 * fp8_qk_norm_rope_bwd: with dn = dy rotated back, xhat = x * rstd, g = dn * w,
 *   dx_j = rstd * (g_j - xhat_j mean_i(g_i xhat_i))   rounded once to x's type
 *   dw_j = sum over tokens and heads of dn_j * xhat_j   fp32, from fp32 sums of
 *          few terms added in 64 bits in a fixed order: same inputs, same bits
 * and dx = dy for values.
 *   dq, dk, dv  device, tokens rows of bf16 words: q_heads, kv_heads, kv_heads
 *               heads; rows dq_stride, dk_stride, dv_stride elements apart
 *   x, wq, ...  as the forward had them
 *   dx          device, tokens x (q_heads + 2 kv_heads) x head_dim of x_dtype,
 *               written
 *   dwq, dwk    device, head_dim floats, written; ignored without weights
 *   ws          device, 16-byte aligned, fp8_qk_norm_rope_bwd_workspace_bytes()
 *               bytes (0 without weights).  The call overwrites it and keeps no
 *               pointer; calls in flight at the same time need separate ones.
 */
int fp8_qk_norm_rope_fwd(const void* x, fp8_dtype_t x_dtype, int64_t x_stride, int64_t tokens, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim, const void* wq, const void* wk, fp8_dtype_t w_dtype,
                         float eps, const int32_t* positions, const float* cos, const float* sin, int32_t rope_rows,
                         int32_t rope_pairs, uint16_t* y, void* stream);
int64_t fp8_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim);
int fp8_qk_norm_rope_bwd(const uint16_t* dq, int64_t dq_stride, const uint16_t* dk, int64_t dk_stride,
                         const uint16_t* dv, int64_t dv_stride, const void* x, fp8_dtype_t x_dtype, int64_t x_stride,
                         int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* wq,
                         const void* wk, fp8_dtype_t w_dtype, float eps, const int32_t* positions, const float* cos,
                         const float* sin, int32_t rope_rows, int32_t rope_pairs, void* dx, float* dwq, float* dwk,
                         void* ws, int64_t ws_bytes, void* stream);

/*
 * Sequences packed one behind the other: sequence i is rows cu_tokens[i] ..
 * cu_tokens[i + 1] - 1 of the token tensors.
 *   cu_tokens  device, batch + 1 int32, ascending, at most `tokens`
 *   max_len    at least every sequence's length (a looser bound may cost empty
 *              workgroups and a worse division of the work)
 * The device array is read by the kernels only.  They stay within the buffers
 * whatever it holds: tokens past max_len or `tokens` do not exist, and rows of
 * outputs that belong to no token of a sequence stay as they are.
 */
typedef struct {
  const int32_t* cu_tokens;
  int32_t batch;
  int32_t tokens;
  int32_t max_len;
  int32_t pad; /* unused */
} fp8_seqs_t;

/*
 * Attention of every token over its own sequence.  Query head a reads key /
 * value head a / (q_heads / kv_heads).  For the query at position p of its
 * sequence:
 *   s_j = scale * sum_d q_d k_jd      over the visible positions j
 *   out = sum_j softmax(s)_j v_j      lse = ln sum_j exp(s_j)
 * Visible: positions of the sequence; causal != 0: j <= p; window > 0:
 * j > p - window (needs causal).  What a query does not see -- other sequences,
 * later tokens, NaN among them -- has no influence on it.  A visible value that
 * is NaN or infinite makes that dimension of the output NaN; NaN and +infinity
 * as a logit, every one.
 *   q, k, v  device, tokens rows of q_heads, kv_heads, kv_heads heads of head_dim
 *            (64, 128 or 256) bf16 words, rows q_stride, k_stride, v_stride
 *            elements apart (slices of one tensor's rows; at most 2^24)
 *   out      device, tokens x q_heads x head_dim bf16 words, written
 *   lse      device, tokens x q_heads floats, written
 * Probabilities are bf16 relative to a running maximum (at most 2^-8 off each, as
 * the values they are multiplied with); logits, sums, maxima and the output are
 * fp32 until the last rounding, lse's last step 64 bits.  Values whose weighted
 * sums pass fp32's range (from some 2^110 on) are out of range.
 * Row pointers and strides (in bytes) must be multiples of 16.  q_heads: a
 * positive multiple of kv_heads (FP8_ERR_SIZE otherwise), scale: finite, and
 * times log2(e) too (likewise).
 *
 * fp8_attention_bwd: with p = exp(s - lse), dp_j = sum_d dout_d v_jd and
 * delta = sum_d dout_d out_d,
 *   ds_j = p_j (dp_j - delta)         dq = scale sum_j ds_j k_j
 *   dk_j = scale sum ds_j q           dv_j = sum p_j dout
 * the sums of dk and dv over the queries that see j, of every head that reads
 * the key head.
 *   dout, out, lse  as the forward wrote them; dout's rows dout_stride apart
 *   dq, dk, dv      device, rows dq_stride, dk_stride, dv_stride elements apart,
 *                   written
 *   ws  device, 16-byte aligned, fp8_attention_bwd_workspace_bytes() bytes.  The
 *       call overwrites it and keeps no pointer; calls in flight at the same
 *       time need separate ones.
 * p and ds are rounded to bf16 as operands of the products; everything else is
 * fp32, rounded once at the end, and nothing is added by atomics (same inputs,
 * same bits).  p is as exact as its argument: beside the logits' own sums, s, lse
 * and their factor log2(e) are rounded to fp32, in all 2^-22 |lse| of p where it
 * counts; a p below 2^-126 is 0.  A query whose out, lse or dout is not finite
 * makes dq of its row, and dk and dv of the keys that it sees, NaN; what is not
 * seen has no influence here either.
 */
int fp8_attention_fwd(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                      int64_t v_stride, const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                      float scale, int32_t causal, int32_t window, uint16_t* out, float* lse, void* stream);
int64_t fp8_attention_bwd_workspace_bytes(const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim);
int fp8_attention_bwd(const uint16_t* dout, int64_t dout_stride, const uint16_t* q, int64_t q_stride,
                      const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const uint16_t* out,
                      const float* lse, const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                      float scale, int32_t causal, int32_t window, uint16_t* dq, int64_t dq_stride, uint16_t* dk,
                      int64_t dk_stride, uint16_t* dv, int64_t dv_stride, void* ws, int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8LIN_TRAIN_H */
