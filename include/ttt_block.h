/*
 * ttt_block.h -- C ABI of the operators a block around the TTT-MLP layer is
 * made of, beside the layer itself (ttt_mlp.h): the residual addition with the
 * root-mean-square norm in front of each part of the block, and linear
 * attention with a decay for each head as its token mixer.  Both have their
 * gradients; the attention has a chunked form for prompts and a recurrent form
 * for the next token(s) of serving sessions.
 *
 * The conventions of ttt_mlp.h hold for every entry point here: device
 * pointers, 16-byte aligned tensors, a 256-byte aligned caller-owned
 * workspace, work enqueued on the caller's stream only, no device memory
 * allocated, no state kept, arguments validated on the host before anything is
 * enqueued, the same status codes, ttt_last_error() and no exceptions.  Every
 * call may be captured into a HIP graph (kernels only, no memset nodes).
 */
#ifndef TTT_BLOCK_H
#define TTT_BLOCK_H

#include "ttt_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Residual addition and root-mean-square norm ----
 *   r = x + res                          (r = x without a residual)
 *   y = r / sqrt(mean_j r_j^2 + eps) * w
 * over `rows` rows of d values.  The sum, the mean of squares and the norm are
 * computed in fp32 from the unrounded sum; r and y are each rounded once (RNE).
 *
 * out = TTT_NORM_FP8 writes y in 8 bits (OCP E4M3) with fp32 scales: for each
 * row, or each run of 128 values of a row, scale = max |y| / 448 (at least
 * 2^-126, and 1 where every y is 0) and the stored value is y / scale, divided in
 * fp32 and rounded to nearest even, so that stored * scale is y.  A NaN is stored
 * as NaN and left out of the maximum; an infinity makes its scale infinite.
 *
 *   rows      1 <= rows < 2^31
 *   d         a multiple of 8, 8 <= d <= 16384
 *   x_stride  values between rows of x (ttt_addnorm_forward) or dy (backward):
 *             a multiple of 8, >= d
 *   y_stride  the same for y or dx (fp8: a multiple of 8 too)
 *   eps       finite, >= 0
 *   dtype     type of x, w and y (unless fp8), dy and dx
 *   res_dtype type of res, r and dr: dtype, or TTT_F32 (a residual stream in
 *             fp32 beside bf16 activations); these tensors are contiguous
 *   out       ttt_norm_out_t
 *   scale_group  fp8 only: 0 (one scale per row) or 128 (d a multiple of 128;
 *             scales [rows][d / 128]) */
typedef enum { TTT_NORM_SAME = 0, TTT_NORM_FP8 = 1 } ttt_norm_out_t;

typedef struct {
  int64_t rows;
  int64_t d;
  int64_t x_stride;
  int64_t y_stride;
  float eps;
  ttt_dtype_t dtype;
  ttt_dtype_t res_dtype;
  ttt_norm_out_t out;
  int32_t scale_group;
} ttt_addnorm_desc_t;

/*   x       [rows][d], rows x_stride apart
 *   res     [rows][d] res_dtype, or NULL (no residual)
 *   w       [d] dtype
 *   r       [rows][d] res_dtype: the sum, for the next addition and the
 *           backward; may be res itself (updated in place); may be NULL
 *   y       [rows][d], rows y_stride apart; may be x itself (same strides,
 *           not fp8)
 *   y_scale fp8: fp32 [rows] or [rows][d / 128]; otherwise NULL */
ttt_status_t ttt_addnorm_forward(const ttt_addnorm_desc_t* desc, const void* x, const void* res,
                                 const void* w, void* r, void* y, float* y_scale, void* stream);

/* Gradients of <dy, y> + <dr_out, r>, with n = r / sqrt(mean r^2 + eps):
 *   dr = (w dy - n mean(w dy n)) / sqrt(mean r^2 + eps) + dr_out
 *   dw = sum over rows of dy n
 * dr is the gradient of x and of res alike.  out must be TTT_NORM_SAME.
 *   dy      [rows][d], rows x_stride apart
 *   r       [rows][d] res_dtype: the forward's r (x when it had no residual)
 *   dr_out  [rows][d] res_dtype: the gradient that reaches r from its other
 *           uses, or NULL
 *   dr      [rows][d] res_dtype; may be dr_out itself
 *   dx      [rows][d] dtype, rows y_stride apart: dr in the activations' type,
 *           or NULL
 *   dw      fp32 [d], or NULL
 *   ws      ttt_addnorm_backward_workspace_size(desc) bytes (partial sums of
 *           dw; may be NULL when dw is)
 * Sums run in an order fixed by the shapes: results are reproducible. */
size_t ttt_addnorm_backward_workspace_size(const ttt_addnorm_desc_t* desc);
ttt_status_t ttt_addnorm_backward(const ttt_addnorm_desc_t* desc, const void* dy, const void* r,
                                  const void* w, const void* dr_out, void* dr, void* dx,
                                  float* dw, void* ws, size_t ws_bytes, void* stream);

/* ---- Linear attention with a decay for each head ----
 * Per sequence and head h, with decay g = exp(log_decay[h]) and a state S
 * [d_key][d_value] that starts from state_in (or 0):
 *   S_t = g S_{t-1} + k_t v_t^T
 *   o_t = scale * q_t S_t
 * which is o_t = scale (sum_{s <= t} g^(t-s) (q_t . k_s) v_s + g^(t+1) q_t S_in).
 * There is no softmax and no denominator; the state has a constant size.  Like
 * the layer's fast weight it is a sum of outer products kept in fp32 per
 * session, one per head and decayed per token.
 *
 *   batch, seq_len  B >= 1 sequences of T tokens, 1 <= T <= 2^30; B H <= 2^21,
 *             B H T <= 2^34
 *   heads     H query heads, 1 <= H <= 65535
 *   kv_heads  G key / value heads, H a multiple of G: query head h reads
 *             key / value head h / (H / G); the state is per query head
 *   d_key, d_value  multiples of 8, 8..128
 *   dtype     of q, k, v, o and the gradients
 *   scale     finite
 *   q_stride, k_stride, v_stride, o_stride  values between sequences, tokens
 *             and heads of q, k, v and o ({batch, token, head}), multiples of 8
 *             and >= 0, token strides of q, k, v and dO at most 2^27 bytes where
 *             there is more than one token: slices of one projection's output can
 *             be passed as they are.  A head's d values are contiguous.  A stride
 *             of 0 in q, k, v or dO repeats a value; o must have no two elements
 *             at one place.  dO has the strides of o; dq, dk and dv are contiguous
 *             [B][T][H or G][d].
 * Shared arguments:
 *   log_decay fp32 [H], on the device: log g, <= 0 in use (0: no decay; -inf: a
 *             token sees itself only)
 *   lengths   int32 [B] on the device, or NULL: sequence b has lengths[b]
 *             tokens (values outside [0, T] are taken as the nearer end); the
 *             rows behind them are not read, their outputs and gradients are 0,
 *             and the state stops at the last token.  A sequence of 0 tokens
 *             keeps its state.
 * States are fp32 [B][H][d_key][d_value], contiguous.  An infinity or NaN reaches
 * only the results that the formula gives it to, and may become NaN there; a
 * token whose decay to a later one is 0 in fp32 may be left out of its result,
 * an infinity or NaN in it too: whether it is depends on the sizes of the call. */
typedef struct {
  int64_t batch;
  int64_t seq_len;
  int64_t heads;
  int64_t kv_heads;
  int64_t d_key;
  int64_t d_value;
  ttt_dtype_t dtype;
  float scale;
  int64_t q_stride[3];
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t o_stride[3];
} ttt_linattn_desc_t;

/* Workspace bytes of ttt_linattn_forward, and of ttt_linattn_backward; the
 * forward's can be 0 (short sequences, or many heads), *bytes is then 0 and ws
 * may be NULL. */
ttt_status_t ttt_linattn_workspace_size(const ttt_linattn_desc_t* desc, size_t* bytes);
ttt_status_t ttt_linattn_backward_workspace_size(const ttt_linattn_desc_t* desc, size_t* bytes);

/*   o          as described by o_stride
 *   state_in   or NULL (0)
 *   state_out  the state behind each sequence's last token; may be state_in
 *              itself (a session's state updated in place); may be NULL
 * Calls of up to 4 tokens run in the recurrent form (state read and
 * written once, all arithmetic in fp32 and o rounded once), longer calls in the
 * chunked form on the matrix cores.  There bf16 operands meet in bf16 products
 * with fp32 accumulation: the decayed scores and the state's copy that meets q are
 * rounded to bf16, so that o is off by up to three roundings (2.0e-3 to 2.4e-3
 * against 64 bits, one rounding is 1.7e-3) where a call of 4 tokens is off by one;
 * the state itself is as exact as fp32 sums (2^-20 over some tens of chunks of 32
 * tokens, 1.4e-7 to 3.6e-7 measured; the roundings of the n chunks, segments or
 * calls that it remembers add like sqrt n, to 1e-6 for 131072 tokens without a decay
 * and 2e-6 for 8192 tokens one by one; the decay's own rounding is not repeated).
 * fp32 operands use fp32 products throughout and round nothing else. */
ttt_status_t ttt_linattn_forward(const ttt_linattn_desc_t* desc, const void* q, const void* k,
                                 const void* v, const float* log_decay, const int32_t* lengths,
                                 const float* state_in, float* state_out, void* o, void* ws,
                                 size_t ws_bytes, void* stream);

/* Gradients of <dO, o> + <dstate_out, S_final>:
 *   dq_t = scale (sum_{s <= t} g^(t-s) (dO_t . v_s) k_s + g^(t+1) S_in dO_t)
 *   dk_s = scale sum_{t >= s} g^(t-s) (v_s . dO_t) q_t + g^(n-1-s) dstate_out v_s
 *   dv_s = scale sum_{t >= s} g^(t-s) (k_s . q_t) dO_t + g^(n-1-s) dstate_out^T k_s
 *   dstate_in = scale sum_t g^(t+1) q_t dO_t^T + g^n dstate_out
 * for a sequence of n tokens; dk and dv are summed over the query heads that
 * share a key / value head (in fp32, in head order).  The decay and the scale
 * are constants of the model and get no gradient.  Any number of tokens runs in
 * the chunked form: with bf16 operands the scores and the copies of S and of its
 * gradient that meet dO, v and k are rounded to bf16 as in the forward, and what
 * is added to the S that only dq's products read carries 16 bits or more (two
 * bf16 terms); dstate_in is as exact as the forward's state.
 *   dO         gradient of o; dstate_out [B][H][d_key][d_value] or NULL (0)
 *   state_in   the forward's, or NULL
 *   dq [B][T][H][d_key], dk [B][T][G][d_key], dv [B][T][G][d_value], dtype
 *   dstate_in  or NULL; may be dstate_out itself */
ttt_status_t ttt_linattn_backward(const ttt_linattn_desc_t* desc, const void* q, const void* k,
                                  const void* v, const float* log_decay, const int32_t* lengths,
                                  const float* state_in, const void* dO, const float* dstate_out,
                                  void* dq, void* dk, void* dv, float* dstate_in, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_BLOCK_H */
