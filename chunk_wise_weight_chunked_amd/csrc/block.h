// block.h -- internal interface between the C ABI (block_api.cpp) and the HIP
// kernels of the block operators (addnorm.hip, linattn.hip).  Not part of the
// public header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer.h"

namespace ttt {

// ------------------------------------------ residual addition + RMS norm
constexpr int64_t kNormMaxD = 16384;
constexpr int kNormScaleGroup = 128;

struct NormArgs {
  int64_t rows, d, x_stride, y_stride;
  float eps;
  Dtype dt, res_dt;
  bool fp8;
  bool grouped;  // fp8: a scale per kNormScaleGroup values instead of per row
};
hipError_t launch_addnorm_forward(const NormArgs& a, const void* x, const void* res, const void* w,
                                  void* r, void* y, float* y_scale, hipStream_t s);
// Partial sums of dw: addnorm_backward_blocks(a) rows of d floats in `part`.
int64_t addnorm_backward_blocks(const NormArgs& a);
hipError_t launch_addnorm_backward(const NormArgs& a, const void* dy, const void* r, const void* w,
                                   const void* dr_out, void* dr, void* dx, float* dw, float* part,
                                   hipStream_t s);

// ------------------------------------------- linear attention with a decay
constexpr int kLinChunk = 32;      // tokens per chunk of the chunked form
constexpr int kLinMaxHead = 128;   // values per head, keys and values
constexpr int kLinStepTokens = 4;  // tokens a call of the recurrent form takes at most

// One [B][T][heads][d] operand; query head h reads head h / rep.
struct LinOperand {
  const void* p;
  int64_t sb, st, sh;  // values between sequences, tokens, heads
  int32_t rep;
};

// o_t = sum_{s <= t} scale_p g^(t-s) (q_t . k_s) v_s + scale_o g^(t+late) q_t S_in,
// S_out = g^n S_in + sum_s scale_u g^(n-s-late) k_s v_s^T over the n tokens of each
// sequence, counted from its last token back when `reverse` is set.  The
// forward has late = 1; the gradients of k and v are the same sums from the
// end with late = 0.
struct LinArgs {
  LinOperand q, k, v;
  void* out;  // [B][T][H][dv] by its strides, rows behind a sequence's end zeroed
  int64_t osb, ost, osh;
  bool out_f32;  // fp32 out whatever the operands' type
  const float* log_decay;
  const int32_t* lengths;  // or null
  const float* s_in;       // [B][H][dk][dv] ([dv][dk] when s_trans), or null
  float* s_out;            // or null
  bool s_trans;
  // bf16: what is added to the state is exact to 24 bits (a state that is given
  // out) instead of 16 (one that only meets bf16 operands).
  bool exact_state;
  int64_t B, T, H, dk, dv;
  float scale_o, scale_p, scale_u;
  int32_t late;
  bool reverse;
  // The segments' states are in the workspace already: left there by
  // launch_linattn_starts, or (seg_trans) for the pass with k and v exchanged
  // (same sequences, lengths and direction).
  bool seg_ready, seg_trans;
  // Two passes in one: this one and the one with (w, v, k) for (q, k, v), whose
  // state is this one's transposed; its outputs go to out2 by their strides.
  bool pair;
  LinOperand w;
  void* out2;
  int64_t osb2, ost2, osh2;
  Dtype dt;
};
// Whether d_key and d_value have tiles of one size: passes with keys and values
// exchanged can then share launches (bf16 passes with LinArgs::pair too).
bool linattn_square(int64_t dk, int64_t dv);
// Bytes of the states that a chunked pass keeps between its launches (0: none).
size_t linattn_segment_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv, Dtype dt);
hipError_t launch_linattn_chunked(const LinArgs& a, float* seg, hipStream_t s);
// The segments' states of one or two passes of the same tiles and exact_state,
// pass i's at i times linattn_segment_bytes behind seg.
hipError_t launch_linattn_starts(const LinArgs* a, int count, float* seg, hipStream_t s);
// The recurrent form, T <= kLinStepTokens (forward direction, late = 1, out in
// the operands' type).
hipError_t launch_linattn_step(const LinArgs& a, hipStream_t s);
// dk [B][T][G][d_key] and dv [B][T][G][d_value] as the sums of their rep query
// heads' parts, [B][G rep][T][d] fp32, in head order.
hipError_t launch_linattn_sum_heads(const float* part_k, void* dk, int64_t d_key,
                                    const float* part_v, void* dv, int64_t d_value, int64_t B,
                                    int64_t T, int64_t G, int64_t rep, Dtype dt, hipStream_t s);

}  // namespace ttt
