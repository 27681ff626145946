// seq.h -- internal interface between the C ABI (seq_api.cpp) and the HIP
// kernels of the sequence operators (embed.hip, gatedrec.hip, act8.hip).  Not
// part of the public header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer.h"

namespace ttt {

// ------------------------------------------------------------- embedding
struct EmbedArgs {
  int64_t N, V, d;
  float scale;
  Dtype dt, out_dt;
  bool wide_ids;  // int64 ids
  bool accumulate;
};
hipError_t launch_embed_forward(const EmbedArgs& a, const void* ids, const void* table, void* out,
                                hipStream_t s);
size_t embed_backward_bytes(const EmbedArgs& a);
hipError_t launch_embed_backward(const EmbedArgs& a, const void* ids, const void* dout, void* grad,
                                 void* ws, hipStream_t s);

// ------------------------------------------------- gated linear recurrence
constexpr int kRecTile = 128;     // tokens of a tile: a state is saved in front of each

// One [B][T][d] operand, channels contiguous.
struct RecOperand {
  const void* p;
  int64_t sb, st;  // values between sequences, tokens
};
struct RecArgs {
  RecOperand x, decay, input;
  RecOperand dh;            // backward
  const float* rate;
  const int32_t* lengths;   // or null
  int64_t B, T, d;
  Dtype dt;
};
size_t gatedrec_forward_bytes(const RecArgs& a);
hipError_t launch_gatedrec_forward(const RecArgs& a, const float* s_in, float* s_out, void* h,
                                   int64_t hsb, int64_t hst, float* saved, void* ws,
                                   hipStream_t s);
size_t gatedrec_backward_bytes(const RecArgs& a);
hipError_t launch_gatedrec_backward(const RecArgs& a, const float* saved, const float* ds_out,
                                    void* dx, void* ddecay, void* dinput, float* drate,
                                    float* ds_in, void* ws, hipStream_t s);

// ------------------------------------------------------ activations in 8 bits
constexpr int kAct8Group = 32;  // values of a row that share a scale
hipError_t launch_act8_store(Dtype dt, const void* x, int64_t rows, int64_t d, int64_t xs,
                             int8_t* codes, uint8_t* exps, hipStream_t s);
hipError_t launch_act8_load(Dtype dt, const int8_t* codes, const uint8_t* exps, int64_t rows,
                            int64_t d, int64_t xs, void* x, hipStream_t s);
struct Act8Grad {
  int64_t rows, d_in, d_out, dys;
  Dtype dt, grad_dt;
  bool accumulate;
};
size_t act8_weight_grad_bytes(const Act8Grad& g);
hipError_t launch_act8_weight_grad(const Act8Grad& g, const int8_t* codes, const uint8_t* exps,
                                   const void* dy, void* grad, void* ws, hipStream_t s);

}  // namespace ttt
