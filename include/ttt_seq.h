/*
 * ttt_seq.h -- C ABI of the operators that a stack of blocks around the TTT-MLP
 * layer (ttt_mlp.h) needs beside those of one block (ttt_block.h): the embedding
 * lookup that makes the layer's X0 and the residual stream from token ids, with
 * the table's gradient; a gated linear recurrence, the token mixer whose decay
 * depends on the token, with its gradients; and activations kept in 8 bits
 * between the forward and the backward pass, with the weight gradient taken from
 * the codes.
 *
 * The conventions of ttt_mlp.h hold for every entry point here: device
 * pointers, 16-byte aligned tensors, a 256-byte aligned caller-owned
 * workspace, work enqueued on the caller's stream only, no device memory
 * allocated, no state kept, arguments validated on the host before anything is
 * enqueued, the same status codes, ttt_last_error() and no exceptions.  Every
 * call may be captured into a HIP graph (kernels only, no memset nodes).  A
 * workspace belongs to one call at a time: calls, or replays of graphs, that
 * may run side by side need one each.  Sums run in an order fixed by the shapes
 * (and the ids): results are reproducible.
 */
#ifndef TTT_SEQ_H
#define TTT_SEQ_H

#include "ttt_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Embedding lookup ----
 *   out[n] = scale * table[ids[n]]              (zeros where ids[n] is outside [0, vocab))
 *   grad[v] (+)= scale * sum over n with ids[n] = v of dout[n]
 * The product and the sum are computed in fp32 and rounded once (RNE).
 *
 *   tokens    1 <= tokens <= 2^28
 *   vocab     rows of the table, 1 <= vocab < 2^31 - 1
 *   d         a multiple of 8, 8 <= d <= 2^20; tokens * d <= 2^38, vocab * d <= 2^40
 *   scale     finite
 *   dtype     type of table, or of dout
 *   out_dtype type of out, or of grad: dtype, or TTT_F32 (an fp32 residual stream,
 *             a gradient held in fp32)
 *   id_bytes  8 (int64 ids) or 4 (int32); ids need the alignment of their type
 *   accumulate  backward: 1 adds to the gradient that is there, 0 writes it whole
 *             (rows without tokens become 0) */
typedef struct {
  int64_t tokens;
  int64_t vocab;
  int64_t d;
  float scale;
  ttt_dtype_t dtype;
  ttt_dtype_t out_dtype;
  int32_t id_bytes;
  int32_t accumulate;
} ttt_embed_desc_t;

/*   ids   [tokens];  table [vocab][d];  out [tokens][d]; all contiguous */
ttt_status_t ttt_embed_forward(const ttt_embed_desc_t* desc, const void* ids, const void* table,
                               void* out, void* stream);

/* The tokens are sorted by id (stably), and the rows of each id added in the order of
 * their places, in pieces of a fixed length: no atomic sums.  Tokens whose id is
 * outside [0, vocab) give nothing.
 *   dout  [tokens][d];  grad [vocab][d]
 *   ws    ttt_embed_backward_workspace_size(desc) bytes (for few tokens 0, ws may then be NULL) */
ttt_status_t ttt_embed_backward_workspace_size(const ttt_embed_desc_t* desc, size_t* bytes);
ttt_status_t ttt_embed_backward(const ttt_embed_desc_t* desc, const void* ids, const void* dout,
                                void* grad, void* ws, size_t ws_bytes, void* stream);

/* ---- Gated linear recurrence ----
 * For each channel, with r = sigmoid(decay_gate), i = sigmoid(input_gate):
 *   a_t = exp(-rate r_t),  b_t = sqrt(1 - a_t^2)
 *   h_t = a_t h_{t-1} + b_t i_t x_t
 * from h = state_in (or 0).  The state is one fp32 value a channel; everything is
 * computed in fp32 (a decay near 1 by its distance from 1, so that long memories
 * lose nothing to its rounding) and h rounded once.  A sigmoid below 2^-126, fp32's
 * smallest normal number (a gate below -87.3), counts as 0.
 *
 *   batch, seq_len  B sequences of T tokens, 1 <= B <= 2^20, T >= 1, B T <= 2^29
 *   d         channels, a multiple of 8, 8 <= d <= 2^20; B d <= 2^28, B T d <= 2^35
 *   dtype     of x, the gates, h and the gradients
 *   x_stride, decay_stride, input_stride, out_stride  values between sequences and
 *             tokens of x, decay_gate, input_gate, and of h (dh in the backward), multiples
 *             of 8, 0 <= stride <= 2^40 (channels contiguous): slices of one projection's
 *             output can be passed as they are.  A stride of 0 in an input repeats a
 *             value; h must have no two elements at one place
 * Shared arguments:
 *   rate     fp32 [d] on the device, >= 0 in use (0: the state is kept and nothing
 *            enters; a negative rate gives NaN)
 *   lengths  int32 [B] on the device, or NULL: sequence b has lengths[b] tokens
 *            (values outside [0, T] are taken as the nearer end); what the rows
 *            behind them hold does not matter, their h and gradients are 0, and the state stops at the last
 *            token.  A sequence of 0 tokens keeps its state.
 * States are fp32 [B][d].  An infinity or NaN stays in its channel, reaches its own
 * token and those that the formula gives it to, and may become NaN there. */
typedef struct {
  int64_t batch;
  int64_t seq_len;
  int64_t d;
  ttt_dtype_t dtype;
  int64_t x_stride[2];
  int64_t decay_stride[2];
  int64_t input_stride[2];
  int64_t out_stride[2];
} ttt_gatedrec_desc_t;

/* Bytes of what the forward can save for the backward (the fp32 state in front of
 * every 128th token, [B][ceil(T / 128)][d]), and of the two workspaces (the forward's
 * can be 0, ws may then be NULL). */
ttt_status_t ttt_gatedrec_saved_size(const ttt_gatedrec_desc_t* desc, size_t* bytes);
ttt_status_t ttt_gatedrec_workspace_size(const ttt_gatedrec_desc_t* desc, size_t* bytes);
ttt_status_t ttt_gatedrec_backward_workspace_size(const ttt_gatedrec_desc_t* desc, size_t* bytes);

/*   state_in   or NULL (0)
 *   state_out  the state behind each sequence's last token; may be state_in itself
 *              (a session's state updated in place); may be NULL
 *   h          as described by out_stride
 *   saved      for the backward, or NULL */
ttt_status_t ttt_gatedrec_forward(const ttt_gatedrec_desc_t* desc, const void* x,
                                  const void* decay_gate, const void* input_gate,
                                  const float* rate, const int32_t* lengths,
                                  const float* state_in, float* state_out, void* h, float* saved,
                                  void* ws, size_t ws_bytes, void* stream);

/* Gradients of <dh, h> + <dstate_out, h_last>.  With l_t = dh_t + a_{t+1} l_{t+1}
 * (dstate_out added to the last token's):
 *   dx_t = l_t b_t i_t,   dinput_t = l_t b_t i_t (1 - i_t) x_t
 *   dz_t = l_t (a_t h_{t-1} - i_t x_t a_t^2 / b_t)
 *   ddecay_t = -dz_t rate r_t (1 - r_t),   drate = -sum_t dz_t r_t
 *   dstate_in = a_1 l_1
 * h is computed again from `saved`, in fp32.  Where b is 0 (a rate of 0, or a decay
 * gate so far down that a is 1) its derivative, which has no bound there, is taken as 0.
 *   saved      the forward's, of the same arguments
 *   dh         gradient of h, by out_stride; dstate_out [B][d] or NULL (0)
 *   dx, ddecay, dinput  [B][T][d] dtype, contiguous
 *   drate      fp32 [d], summed over all tokens
 *   dstate_in  fp32 [B][d], or NULL; may be dstate_out itself */
ttt_status_t ttt_gatedrec_backward(const ttt_gatedrec_desc_t* desc, const void* x,
                                   const void* decay_gate, const void* input_gate,
                                   const float* rate, const int32_t* lengths, const float* saved,
                                   const void* dh, const float* dstate_out, void* dx,
                                   void* ddecay, void* dinput, float* drate, float* dstate_in,
                                   void* ws, size_t ws_bytes, void* stream);

/* ---- Activations in 8 bits ----
 * Each run of 32 values of a row (the last one of a row may be shorter) shares the
 * smallest power of two 2^e, -126 <= e <= 121, that takes its largest value to at most 127:
 *   code = round(x / 2^e) (RNE, at most 127 at the end of fp32's range), exps = e + 127
 *   x8 = code * 2^e
 * so that x8 is off by at most max |x| / 127 (2^-127 for the smallest), finite where x is, and
 * exact in bf16.
 * A run with an infinity or a NaN has exps = 255 and stands for NaN.
 *   rows     1 <= rows < 2^31
 *   d        a multiple of 8, 8 <= d <= 2^20; rows * d <= 2^40
 *   x_stride values between rows of x: a multiple of 8, d <= x_stride <= 2^40
 *   dtype    of x
 *   codes int8 [rows][d], exps uint8 [rows][ceil(d / 32)], contiguous; exps needs no
 *   alignment */
typedef struct {
  int64_t rows;
  int64_t d;
  int64_t x_stride;
  ttt_dtype_t dtype;
} ttt_act8_desc_t;
ttt_status_t ttt_act8_store(const ttt_act8_desc_t* desc, const void* x, int8_t* codes,
                            uint8_t* exps, void* stream);
ttt_status_t ttt_act8_load(const ttt_act8_desc_t* desc, const int8_t* codes, const uint8_t* exps,
                           void* x, void* stream);

/* The gradient of a weight [d_in][d_out] from the activations kept in front of it:
 *   grad (+)= x8^T dy
 * On the bf16 matrix cores: every product of x8 and a bf16 dy is exact; an fp32 dy is taken
 * as the three bf16 values whose sum it is (what it has below multiples of 2^-133, the
 * smallest of bf16, is left out: values below 2^-109 alone have that).  Sums are fp32,
 * rounded once.
 *   rows, d_in  as rows and d above; rows * d_in and rows * d_out <= 2^40
 *   d_out    a multiple of 8, 8 <= d_out <= 2^20; d_in * d_out <= 2^36
 *   dy_stride  values between rows of dy: a multiple of 8, d_out <= dy_stride <= 2^20
 *   dtype    of dy;  grad_dtype: dtype or TTT_F32
 *   accumulate  1: adds to the gradient that is there (TTT_F32 only) */
typedef struct {
  int64_t rows;
  int64_t d_in;
  int64_t d_out;
  int64_t dy_stride;
  ttt_dtype_t dtype;
  ttt_dtype_t grad_dtype;
  int32_t accumulate;
} ttt_act8_wgrad_desc_t;
ttt_status_t ttt_act8_weight_grad_workspace_size(const ttt_act8_wgrad_desc_t* desc, size_t* bytes);
ttt_status_t ttt_act8_weight_grad(const ttt_act8_wgrad_desc_t* desc, const int8_t* codes,
                                  const uint8_t* exps, const void* dy, void* grad, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_SEQ_H */
