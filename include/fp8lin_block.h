/*
 * fp8lin -- the operators of a transformer block around the FP8-AMAX linear
 * layer (fp8lin.h), in the same library (libfp8lin.so):
 *   - the RMS norm with the residual's addition in front of a product, with an
 *     output in FP8 codes, and its backward pass;
 *   - a paged cache of keys and values in FP8 with one scale for each block of
 *     tokens and head: written with the rotary positions applied, read back,
 *     and attended to.
 * Formats, dtypes, status codes and the conventions for every entry point are
 * fp8lin.h's.  Scales are its power-of-two biases: a code c stands for
 * value(c) * 2^-bias.
 */
#ifndef FP8LIN_BLOCK_H
#define FP8LIN_BLOCK_H

#include "fp8lin.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * RMS norm with the residual's addition.
 *   h = round(x + residual)      rounded to the residual's type; without a
 *                                residual h = x and nothing is written
 *   rstd = (mean_j h_j^2 + eps)^(-1/2)      per row, fp32
 *   y_j = (h_j * rstd) * w_j                fp32, then rounded once
 * h is rounded before it is squared, so that the backward pass, which reads
 * the stored h, is the gradient of this function.  A row whose squares
 * overflow fp32 gives rstd = 0; NaN and infinities follow IEEE arithmetic.
 *   x         device, rows x d of x_dtype
 *   residual  device, rows x d of r_dtype, or NULL
 *   w         device, d values of w_dtype
 *   h         device, rows x d of r_dtype, written (may be the residual
 *             itself); required with a residual, ignored without one
 *   rstd      device, rows floats, written; optional but for
 *             fp8_rmsnorm_quantize
 * Tensors need 16-byte alignment, rstd and the words below 4.  1 <= d <= 32768,
 * or 16384 where d is not a multiple of 4 (FP8_ERR_SIZE otherwise: a row stays
 * in registers); rows >= 0.
 *
 * fp8_rmsnorm_fwd: y in bf16.
 *   y_amax  device float, optional: max |y| of the rounded outputs, bits as
 *           fp8_amax over y (0 for no rows), so fp8_compute_bias can follow.
 *
 * fp8_rmsnorm_cast: the codes of y at a given bias, fp8_scale_cast's rounding
 * ("Proposed method", bullets 3-4, fused with the norm): a scale calibrated
 * beforehand, or delayed scaling with the bias of the previous step's amax.
 *   bias    device int32
 *   fmt     FP8_E4M3 or FP8_E5M2 (FP8_ERR_FORMAT otherwise)
 *   y_amax  device float, optional: max |y| of the fp32 values
 * Both take one launch, and a one-lane clear where y_amax is given.
 *
 * fp8_rmsnorm_quantize: current scaling -- the tensor's amax, its bias (as
 * fp8_compute_bias at `margin`) and the codes.  One launch for one row; two
 * for more: the first writes h, rstd and every row's amax, the second forms y
 * again from them.  Same inputs, same bits; nothing is accumulated by atomics.
 *   row_amax  device, rows floats, written with max |y| of each row
 *   amax      device float, bias  device int32, written (0, 0 for no rows)
 */
int fp8_rmsnorm_fwd(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype,
                    const void* w, fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h,
                    float* rstd, uint16_t* y, float* y_amax, void* stream);
int fp8_rmsnorm_cast(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype,
                     const void* w, fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h,
                     float* rstd, const int32_t* bias, fp8_format_t fmt, uint8_t* y, float* y_amax,
                     void* stream);
int fp8_rmsnorm_quantize(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype,
                         const void* w, fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h,
                         float* rstd, fp8_format_t fmt, int32_t margin, uint8_t* y, float* row_amax,
                         float* amax, int32_t* bias, void* stream);

/*
 * Backward pass of the norm: with g = dy * w, xhat = h * rstd and
 * c = mean_j g_j xhat_j,
 *   dx_j = rstd * (g_j - xhat_j * c) + dh_j     rounded once to h's type
 *   dw_j = sum over rows of dy_j * xhat_j       fp32
 * dx is the gradient of x and of the residual alike.
 *   dy    device, rows x d of dy_dtype (a data-gradient product's fp32 output,
 *         or bf16)
 *   h     device, rows x d of h_dtype: the forward's h (x without a residual)
 *   rstd  device, rows floats of the forward
 *   dh    device, rows x d of h_dtype, optional: the gradient that reaches h
 *         past the norm
 *   dx    device, rows x d of h_dtype, written (may be dh itself)
 *   dw    device, d floats, written (zeros for no rows)
 *   dx_amax  device float, optional: max |dx| of the rounded outputs
 *   ws    device, 16-byte aligned, fp8_rmsnorm_bwd_workspace_bytes(rows, d)
 *         bytes: partial sums of dw, added in a fixed order (same inputs, same
 *         bits).  The call overwrites it and keeps no pointer.
 * d as above.
 */
int64_t fp8_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t d);
int fp8_rmsnorm_bwd(const void* dy, fp8_dtype_t dy_dtype, const void* h, fp8_dtype_t h_dtype,
                    const void* w, fp8_dtype_t w_dtype, const float* rstd, const void* dh, int64_t rows,
                    int64_t d, void* dx, float* dw, float* dx_amax, void* ws, int64_t ws_bytes,
                    void* stream);

/*
 * A paged cache of keys and values in FP8.  Blocks of `block_size` tokens are
 * dealt out by the caller through a block table; each block and head has one
 * bias for its keys and one for its values.  Keys lie token by token; values
 * lie transposed, the tokens of one head dimension side by side, which is the
 * order the product of the probabilities with the values consumes them in.
 *   k       [num_blocks][heads][block_size][head_dim] codes
 *   v       [num_blocks][heads][head_dim][block_size] codes
 *   k_bias, v_bias  [num_blocks][heads]
 * All device memory, codes 16-byte aligned, biases 4.  block_size 16, 32, 64
 * or 128; head_dim 64, 128 or 256; fmt FP8_E4M3 or FP8_E5M2; heads and
 * num_blocks >= 1.
 */
#define FP8_KV_MAX_BIAS 126 /* largest bias of a block, and that of one of zeros only */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  int32_t* k_bias;
  int32_t* v_bias;
  int32_t num_blocks;
  int32_t heads;
  int32_t block_size;
  int32_t head_dim;
  int32_t fmt; /* fp8_format_t */
  int32_t pad; /* unused */
} fp8_kv_cache_t;

/*
 * A ragged batch of sequences.  Sequence i has lens[i] tokens in the cache,
 * the last n_i = cu_tokens[i + 1] - cu_tokens[i] of them new: rows
 * cu_tokens[i] .. cu_tokens[i + 1] - 1 of the packed token tensors, at
 * positions lens[i] - n_i .. lens[i] - 1.  Its token at position p lies in
 * block block_table[i][p / block_size], slot p % block_size.
 *   cu_tokens    device, batch + 1 int32, ascending from 0 to `tokens`
 *   lens         device, batch int32
 *   block_table  device, batch x table_width int32
 *   tokens       rows of the packed tensors
 *   max_new      at least every n_i (a looser bound costs nothing past `tokens`
 *                and max_len);  max_len  at least every lens[i], at most
 *                table_width * block_size and 2^30 (FP8_ERR_SIZE otherwise)
 * The device arrays are read by the kernels only.  They stay within the
 * buffers whatever the arrays hold: a table entry outside 0 .. num_blocks - 1
 * is a block that is neither written nor seen, tokens past max_new, max_len or
 * `tokens` do not exist, and rows of outputs that belong to no token of a
 * sequence stay as they are.
 */
typedef struct {
  const int32_t* cu_tokens;
  const int32_t* lens;
  const int32_t* block_table;
  int32_t batch;
  int32_t table_width;
  int32_t tokens;
  int32_t max_new;
  int32_t max_len;
  int32_t pad; /* unused */
} fp8_kv_batch_t;

/*
 * Writes the batch's new keys and values into the cache, in one launch.
 *   k, v    device, tokens rows of heads x head_dim values of `dtype`, rows
 *           k_stride / v_stride elements apart (a slice of the fused query /
 *           key / value product's rows)
 *   q       device, optional: tokens rows of q_heads x head_dim, q_stride
 *           apart, of `dtype`; q_out  device, tokens x q_heads x head_dim bf16
 *           words: the (rotated) queries, rounded to nearest even
 *   cos, sin  device, rope_rows x head_dim / 2 floats, or both NULL (keys and
 *           queries are not rotated).  Row p holds position p; rope_rows >=
 *           max_len.  rope_pairs 0: dimension j rotates with j + head_dim / 2;
 *           1: dimension 2j with 2j + 1.  (a, b) -> (a cos - b sin,
 *           b cos + a sin), each product and the sum rounded to fp32.
 * Scales: in each touched block and head, A = the largest finite magnitude of
 * the new keys (rotated), and b = the largest integer with A * 2^b <= the
 * format's maximum, at most FP8_KV_MAX_BIAS (also for A = 0).  Where the block
 * already held tokens of the sequence (the first new one has slot > 0) b is
 * at most the block's bias, and if it is below it, those tokens are coded
 * again at b -- a power of two apart, so their codes change by rounding only
 * where they become subnormal (codes of NaN and infinity stay).  Infinities
 * saturate, NaN gets the NaN code; neither moves the scale.  Values likewise, without rotation.
 * Writing the same tokens again changes nothing.  A block may be shared by
 * several sequences only while none writes into it.
 * Row pointers and strides (in bytes) must be multiples of 16
 * (FP8_ERR_ALIGN).  FP8_ERR_SIZE also for more than 2^31 - 1 workgroups:
 * batch * ((max_new - 1) / block_size + 2) * heads * 2 + batch * max_new.
 */
int fp8_kv_append(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, const void* k,
                  int64_t k_stride, const void* v, int64_t v_stride, fp8_dtype_t dtype, const void* q,
                  int64_t q_stride, int32_t q_heads, uint16_t* q_out, const float* cos, const float* sin,
                  int32_t rope_rows, int32_t rope_pairs, void* stream);

/*
 * Reads the batch's last n_i tokens of every sequence back (n_i = lens[i]: the
 * whole sequence), each value(code) * 2^-bias rounded once to out_dtype.
 *   k_out, v_out  device, tokens x heads x head_dim of out_dtype, 16-byte
 *                 aligned, written; either may be NULL.  Rows of tokens whose
 *                 block is not in the cache become zeros.
 */
int fp8_kv_read(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, fp8_dtype_t out_dtype,
                void* k_out, void* v_out, void* stream);

/*
 * Attention of the batch's new tokens over their sequences in the cache (which
 * already holds the new tokens themselves).  Query head a reads key / value
 * head a / (q_heads / heads).  For the query at position p:
 *   s_j = scale * sum_d q_d k_jd      over the visible positions j
 *   out = sum_j softmax(s)_j v_j      lse = ln sum_j exp(s_j)
 * Visible: j < lens[i]; causal != 0: j <= p; window > 0: j > p - window
 * (needs causal).  A query that sees nothing gets out = 0 and lse = -inf;
 * what lies in invisible slots -- NaN codes among it -- has no influence.  A
 * visible value whose code is NaN or (E5M2) an infinity makes that dimension of
 * the output NaN, whatever its weight; NaN and +infinity as a logit, every one.
 *   q     device, tokens rows of q_heads x head_dim bf16 words, q_stride
 *         elements apart (rows multiples of 16 bytes)
 *   out   device, tokens x q_heads x head_dim bf16 words, written
 *   lse   device, tokens x q_heads floats, written; optional
 *   ws    device, 16-byte aligned, fp8_kv_attention_workspace_bytes() bytes
 *         (0: none needed): partial results of long sequences, split so that a
 *         few queries fill the chip; joined in a fixed order (same inputs,
 *         same bits).  Calls in flight at the same time need separate ones.
 * Keys widen exactly to bf16; values to fp16, scaled by the smallest bias met so
 * far among the blocks that a workgroup's queries read, seen or not: exactly,
 * but for what lies below 2^-40 of the largest value of that bias (E4M3 blocks
 * within 22 of it are exact, E5M2 ones within 8, their larger codes within
 * 30).  Probabilities are fp16 relative to a running maximum; logits, sums,
 * maxima and the join are fp32, lse's last step 64 bits.
 * q_heads: a positive multiple of heads (FP8_ERR_SIZE otherwise, and where
 * max_new * q_heads / heads passes 2^31 - 129).
 */
int64_t fp8_kv_attention_workspace_bytes(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch,
                                         int32_t q_heads);
int fp8_kv_attention(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, const uint16_t* q,
                     int64_t q_stride, int32_t q_heads, float scale, int32_t causal, int32_t window,
                     uint16_t* out, float* lse, void* ws, int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8LIN_BLOCK_H */
