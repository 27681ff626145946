// seq_api.cpp -- C ABI of the sequence operators (include/ttt_seq.h): validation,
// workspace sizes and the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ttt_seq.h"
#include "api_common.h"
#include "seq.h"

using namespace ttt::api;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxWidth = (int64_t)1 << 20;

bool over(int64_t a, int64_t b, int bits) { return (__int128)a * b > ((__int128)1 << bits); }

ttt_status_t check_width(const char* name, int64_t d) {
  if (d < 1) return fail(TTT_ERR_INVALID_ARGUMENT, "%s must be >= 1", name);
  if (d % 8 || d > kMaxWidth)
    return fail(TTT_ERR_UNSUPPORTED, "%s must be a multiple of 8, at most 2^20", name);
  return TTT_OK;
}

// ---------------------------------------------------------------- embedding
ttt_status_t embed_args(const ttt_embed_desc_t* d, ttt::EmbedArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->tokens < 1 || d->vocab < 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "tokens and vocab must be >= 1");
  if (d->tokens > ((int64_t)1 << 28)) return fail(TTT_ERR_UNSUPPORTED, "tokens must be <= 2^28");
  if (d->vocab >= ((int64_t)1 << 31) - 1) return fail(TTT_ERR_UNSUPPORTED, "vocab must be < 2^31 - 1");
  if (ttt_status_t st = check_width("d", d->d)) return st;
  if (over(d->tokens, d->d, 38) || over(d->vocab, d->d, 40))
    return fail(TTT_ERR_UNSUPPORTED, "tokens * d must be <= 2^38 and vocab * d <= 2^40");
  if (!std::isfinite(d->scale)) return fail(TTT_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  if (d->out_dtype != d->dtype && d->out_dtype != TTT_F32)
    return fail(TTT_ERR_INVALID_ARGUMENT, "out_dtype must be dtype or TTT_F32");
  if (d->id_bytes != 4 && d->id_bytes != 8)
    return fail(TTT_ERR_INVALID_ARGUMENT, "id_bytes must be 4 or 8");
  if (d->accumulate != 0 && d->accumulate != 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
  *a = ttt::EmbedArgs{d->tokens, d->vocab, d->d, d->scale, to_dtype(d->dtype),
                      to_dtype(d->out_dtype), d->id_bytes == 8, d->accumulate != 0};
  return TTT_OK;
}

// The call's ids beside its other buffers.
ttt_status_t check_ids(const BufferList& b, const ttt_embed_desc_t* d, const void* ids) {
  if (!aligned(ids, d->id_bytes))
    return fail(TTT_ERR_INVALID_ARGUMENT, "ids must be %d-byte aligned", (int)d->id_bytes);
  if (ttt_status_t st = b.check()) return st;
  return b.check_against(range("ids", ids, (size_t)d->tokens * d->id_bytes));
}

// ----------------------------------------------------- gated linear recurrence
ttt_status_t rec_args(const ttt_gatedrec_desc_t* d, ttt::RecArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->batch < 1 || d->seq_len < 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "batch and seq_len must be >= 1");
  if (ttt_status_t st = check_width("d", d->d)) return st;
  // what one launch holds: tiles of 128 tokens and 64 channels, 256 threads each
  if (d->batch > ((int64_t)1 << 20) || over(d->batch, d->seq_len, 29) || over(d->batch, d->d, 28) ||
      over(d->batch * std::min<int64_t>(d->seq_len, (int64_t)1 << 30), d->d, 35))
    return fail(TTT_ERR_UNSUPPORTED,
                "batch must be <= 2^20, batch * seq_len <= 2^29, batch * d <= 2^28 and batch * "
                "seq_len * d <= 2^35");
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  for (const int64_t* st : {d->x_stride, d->decay_stride, d->input_stride, d->out_stride})
    for (int i = 0; i < 2; ++i) {
      if (st[i] < 0) return fail(TTT_ERR_INVALID_ARGUMENT, "strides must be >= 0");
      if (st[i] % 8 || st[i] > kMaxStride)
        return fail(TTT_ERR_UNSUPPORTED, "strides must be multiples of 8, at most 2^40");
    }
  for (const int64_t* st : {d->x_stride, d->decay_stride, d->input_stride, d->out_stride})
    if ((__int128)st[0] * (d->batch - 1) + (__int128)st[1] * (d->seq_len - 1) > ((__int128)1 << 56))
      return fail(TTT_ERR_UNSUPPORTED, "a tensor must span less than 2^56 values");
  *a = ttt::RecArgs{};
  a->B = d->batch, a->T = d->seq_len, a->d = d->d, a->dt = to_dtype(d->dtype);
  return TTT_OK;
}

size_t rec_bytes(const ttt_gatedrec_desc_t* d, const int64_t st[2]) {
  return (size_t)(st[0] * (d->batch - 1) + st[1] * (d->seq_len - 1) + d->d) *
         ttt::dtype_bytes(to_dtype(d->dtype));
}
size_t rec_state_bytes(const ttt_gatedrec_desc_t* d) {
  return (size_t)(d->batch * d->d) * sizeof(float);
}
size_t rec_saved_bytes(const ttt_gatedrec_desc_t* d) {
  return rec_state_bytes(d) * (size_t)((d->seq_len + ttt::kRecTile - 1) / ttt::kRecTile);
}

// Whether h has one place for each element.
bool one_place_each(const ttt_gatedrec_desc_t* d) {
  std::pair<int64_t, int64_t> x[2] = {{d->out_stride[0], d->batch}, {d->out_stride[1], d->seq_len}};
  std::sort(x, x + 2);
  __int128 extent = d->d;
  for (const auto& [stride, size] : x) {
    if (size == 1) continue;
    if (stride < extent) return false;
    extent += (__int128)stride * (size - 1);
  }
  return true;
}

// What both directions read besides their states.
void rec_inputs(const ttt_gatedrec_desc_t* d, BufferList* b, ttt::RecArgs* a, const void* x,
                const void* decay, const void* input, const float* rate, const int32_t* lengths) {
  b->in("x", x, rec_bytes(d, d->x_stride));
  b->in("decay_gate", decay, rec_bytes(d, d->decay_stride));
  b->in("input_gate", input, rec_bytes(d, d->input_stride));
  b->in("rate", rate, d->d * sizeof(float));
  a->x = {x, d->x_stride[0], d->x_stride[1]};
  a->decay = {decay, d->decay_stride[0], d->decay_stride[1]};
  a->input = {input, d->input_stride[0], d->input_stride[1]};
  a->rate = rate, a->lengths = lengths;
}

ttt_status_t rec_check(const ttt_gatedrec_desc_t* d, const BufferList& b, const int32_t* lengths) {
  if (!aligned(lengths, 4))
    return fail(TTT_ERR_INVALID_ARGUMENT, "lengths must be 4-byte aligned");
  if (ttt_status_t st = b.check()) return st;
  return b.check_against(range("lengths", lengths, lengths ? d->batch * sizeof(int32_t) : 0));
}

// ---------------------------------------------------------- activations in 8 bits
ttt_status_t act8_dims(const ttt_act8_desc_t* d) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 1) return fail(TTT_ERR_INVALID_ARGUMENT, "rows must be >= 1");
  if (d->rows > INT32_MAX) return fail(TTT_ERR_UNSUPPORTED, "rows must be < 2^31");
  if (ttt_status_t st = check_width("d", d->d)) return st;
  if (over(d->rows, d->d, 40)) return fail(TTT_ERR_UNSUPPORTED, "rows * d must be <= 2^40");
  if (d->x_stride < d->d) return fail(TTT_ERR_INVALID_ARGUMENT, "x_stride must be >= d");
  if (d->x_stride % 8 || d->x_stride > kMaxStride)
    return fail(TTT_ERR_UNSUPPORTED, "x_stride must be a multiple of 8, at most 2^40");
  if (over(d->rows, d->x_stride, 56))
    return fail(TTT_ERR_UNSUPPORTED, "a tensor must span less than 2^56 values");
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  return TTT_OK;
}
size_t act8_x_bytes(const ttt_act8_desc_t* d) {
  return (size_t)((d->rows - 1) * d->x_stride + d->d) * ttt::dtype_bytes(to_dtype(d->dtype));
}
size_t exps_bytes(int64_t rows, int64_t d) {
  return (size_t)rows * ((d + ttt::kAct8Group - 1) / ttt::kAct8Group);
}

ttt_status_t act8_grad_args(const ttt_act8_wgrad_desc_t* d, ttt::Act8Grad* g) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 1) return fail(TTT_ERR_INVALID_ARGUMENT, "rows must be >= 1");
  if (d->rows > INT32_MAX) return fail(TTT_ERR_UNSUPPORTED, "rows must be < 2^31");
  if (ttt_status_t st = check_width("d_in", d->d_in)) return st;
  if (ttt_status_t st = check_width("d_out", d->d_out)) return st;
  if (over(d->rows, d->d_in, 40) || over(d->rows, d->d_out, 40) || over(d->d_in, d->d_out, 36))
    return fail(TTT_ERR_UNSUPPORTED,
                "rows * d_in and rows * d_out must be <= 2^40 and d_in * d_out <= 2^36");
  if (d->dy_stride < d->d_out) return fail(TTT_ERR_INVALID_ARGUMENT, "dy_stride must be >= d_out");
  if (d->dy_stride % 8 || d->dy_stride > kMaxWidth)
    return fail(TTT_ERR_UNSUPPORTED, "dy_stride must be a multiple of 8, at most 2^20");
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  if (d->grad_dtype != d->dtype && d->grad_dtype != TTT_F32)
    return fail(TTT_ERR_INVALID_ARGUMENT, "grad_dtype must be dtype or TTT_F32");
  if (d->accumulate != 0 && d->accumulate != 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
  if (d->accumulate && d->grad_dtype != TTT_F32)
    return fail(TTT_ERR_INVALID_ARGUMENT, "accumulate needs grad_dtype = TTT_F32");
  *g = ttt::Act8Grad{d->rows, d->d_in, d->d_out, d->dy_stride, to_dtype(d->dtype),
                     to_dtype(d->grad_dtype), d->accumulate != 0};
  return TTT_OK;
}

}  // namespace

extern "C" {

ttt_status_t ttt_embed_forward(const ttt_embed_desc_t* desc, const void* ids, const void* table,
                               void* out, void* stream) {
  ttt::EmbedArgs a;
  if (ttt_status_t st = embed_args(desc, &a)) return st;
  if (!ids || !table || !out)
    return fail(TTT_ERR_INVALID_ARGUMENT, "ids, table and out must be non-NULL");
  BufferList b;
  b.in("table", table, (size_t)(a.V * a.d) * ttt::dtype_bytes(a.dt));
  b.out("out", out, (size_t)(a.N * a.d) * ttt::dtype_bytes(a.out_dt));
  if (ttt_status_t st = check_ids(b, desc, ids)) return st;
  const hipError_t e = ttt::launch_embed_forward(a, ids, table, out, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "embed_forward");
}

ttt_status_t ttt_embed_backward_workspace_size(const ttt_embed_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  ttt::EmbedArgs a;
  if (ttt_status_t st = embed_args(desc, &a)) return st;
  *bytes = ttt::embed_backward_bytes(a);
  return ok();
}

ttt_status_t ttt_embed_backward(const ttt_embed_desc_t* desc, const void* ids, const void* dout,
                                void* grad, void* ws, size_t ws_bytes, void* stream) {
  ttt::EmbedArgs a;
  if (ttt_status_t st = embed_args(desc, &a)) return st;
  if (!ids || !dout || !grad)
    return fail(TTT_ERR_INVALID_ARGUMENT, "ids, dout and grad must be non-NULL");
  const size_t need = ttt::embed_backward_bytes(a);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  BufferList b;
  b.in("dout", dout, (size_t)(a.N * a.d) * ttt::dtype_bytes(a.dt));
  b.out("grad", grad, (size_t)(a.V * a.d) * ttt::dtype_bytes(a.out_dt));
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = check_ids(b, desc, ids)) return st;
  const hipError_t e =
      ttt::launch_embed_backward(a, ids, dout, grad, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "embed_backward");
}

ttt_status_t ttt_gatedrec_saved_size(const ttt_gatedrec_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  ttt::RecArgs a;
  if (ttt_status_t st = rec_args(desc, &a)) return st;
  *bytes = rec_saved_bytes(desc);
  return ok();
}

ttt_status_t ttt_gatedrec_workspace_size(const ttt_gatedrec_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  ttt::RecArgs a;
  if (ttt_status_t st = rec_args(desc, &a)) return st;
  *bytes = ttt::gatedrec_forward_bytes(a);
  return ok();
}

ttt_status_t ttt_gatedrec_backward_workspace_size(const ttt_gatedrec_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  ttt::RecArgs a;
  if (ttt_status_t st = rec_args(desc, &a)) return st;
  *bytes = ttt::gatedrec_backward_bytes(a);
  return ok();
}

ttt_status_t ttt_gatedrec_forward(const ttt_gatedrec_desc_t* desc, const void* x,
                                  const void* decay_gate, const void* input_gate,
                                  const float* rate, const int32_t* lengths,
                                  const float* state_in, float* state_out, void* h, float* saved,
                                  void* ws, size_t ws_bytes, void* stream) {
  ttt::RecArgs a;
  if (ttt_status_t st = rec_args(desc, &a)) return st;
  if (!x || !decay_gate || !input_gate || !rate || !h)
    return fail(TTT_ERR_INVALID_ARGUMENT, "x, decay_gate, input_gate, rate and h must be non-NULL");
  if (!one_place_each(desc))
    return fail(TTT_ERR_INVALID_ARGUMENT, "out_stride gives two elements of h one place");
  const size_t need = ttt::gatedrec_forward_bytes(a);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  BufferList b;
  rec_inputs(desc, &b, &a, x, decay_gate, input_gate, rate, lengths);
  b.in("state_in", state_in, rec_state_bytes(desc));
  b.out("h", h, rec_bytes(desc, desc->out_stride));
  b.out("state_out", state_out, rec_state_bytes(desc), state_in);
  b.out("saved", saved, rec_saved_bytes(desc));
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = rec_check(desc, b, lengths)) return st;
  const hipError_t e =
      ttt::launch_gatedrec_forward(a, state_in, state_out, h, desc->out_stride[0],
                                   desc->out_stride[1], saved, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gatedrec_forward");
}

ttt_status_t ttt_gatedrec_backward(const ttt_gatedrec_desc_t* desc, const void* x,
                                   const void* decay_gate, const void* input_gate,
                                   const float* rate, const int32_t* lengths, const float* saved,
                                   const void* dh, const float* dstate_out, void* dx,
                                   void* ddecay, void* dinput, float* drate, float* dstate_in,
                                   void* ws, size_t ws_bytes, void* stream) {
  ttt::RecArgs a;
  if (ttt_status_t st = rec_args(desc, &a)) return st;
  if (!x || !decay_gate || !input_gate || !rate || !saved || !dh || !dx || !ddecay || !dinput ||
      !drate)
    return fail(TTT_ERR_INVALID_ARGUMENT,
                "x, decay_gate, input_gate, rate, saved, dh, dx, ddecay, dinput and drate must be "
                "non-NULL");
  const size_t need = ttt::gatedrec_backward_bytes(a);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  const size_t n = (size_t)(a.B * a.T * a.d) * ttt::dtype_bytes(a.dt);
  BufferList b;
  rec_inputs(desc, &b, &a, x, decay_gate, input_gate, rate, lengths);
  b.in("saved", saved, rec_saved_bytes(desc));
  b.in("dh", dh, rec_bytes(desc, desc->out_stride));
  b.in("dstate_out", dstate_out, rec_state_bytes(desc));
  b.out("dx", dx, n);
  b.out("ddecay", ddecay, n);
  b.out("dinput", dinput, n);
  b.out("drate", drate, a.d * sizeof(float));
  b.out("dstate_in", dstate_in, rec_state_bytes(desc), dstate_out);
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = rec_check(desc, b, lengths)) return st;
  a.dh = {dh, desc->out_stride[0], desc->out_stride[1]};
  const hipError_t e =
      ttt::launch_gatedrec_backward(a, saved, dstate_out, dx, ddecay, dinput, drate, dstate_in, ws,
                                    static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "gatedrec_backward");
}

ttt_status_t ttt_act8_store(const ttt_act8_desc_t* desc, const void* x, int8_t* codes,
                            uint8_t* exps, void* stream) {
  if (ttt_status_t st = act8_dims(desc)) return st;
  if (!x || !codes || !exps)
    return fail(TTT_ERR_INVALID_ARGUMENT, "x, codes and exps must be non-NULL");
  BufferList b;
  b.in("x", x, act8_x_bytes(desc));
  b.out("codes", codes, (size_t)(desc->rows * desc->d));
  if (ttt_status_t st = b.check()) return st;
  const Range e8 = range("exps", exps, exps_bytes(desc->rows, desc->d));
  for (const auto& i : {b.items[0], b.items[1]})
    if (overlaps(e8, i.r))
      return fail(TTT_ERR_INVALID_ARGUMENT, "exps overlaps %s", i.r.name);
  const hipError_t e =
      ttt::launch_act8_store(to_dtype(desc->dtype), x, desc->rows, desc->d, desc->x_stride, codes,
                             exps, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "act8_store");
}

ttt_status_t ttt_act8_load(const ttt_act8_desc_t* desc, const int8_t* codes, const uint8_t* exps,
                           void* x, void* stream) {
  if (ttt_status_t st = act8_dims(desc)) return st;
  if (!x || !codes || !exps)
    return fail(TTT_ERR_INVALID_ARGUMENT, "x, codes and exps must be non-NULL");
  BufferList b;
  b.in("codes", codes, (size_t)(desc->rows * desc->d));
  b.out("x", x, act8_x_bytes(desc));
  if (ttt_status_t st = b.check()) return st;
  if (ttt_status_t st =
          b.check_against(range("exps", exps, exps_bytes(desc->rows, desc->d))))
    return st;
  const hipError_t e =
      ttt::launch_act8_load(to_dtype(desc->dtype), codes, exps, desc->rows, desc->d, desc->x_stride,
                            x, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "act8_load");
}

ttt_status_t ttt_act8_weight_grad_workspace_size(const ttt_act8_wgrad_desc_t* desc,
                                                 size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  ttt::Act8Grad g;
  if (ttt_status_t st = act8_grad_args(desc, &g)) return st;
  *bytes = ttt::act8_weight_grad_bytes(g);
  return ok();
}

ttt_status_t ttt_act8_weight_grad(const ttt_act8_wgrad_desc_t* desc, const int8_t* codes,
                                  const uint8_t* exps, const void* dy, void* grad, void* ws,
                                  size_t ws_bytes, void* stream) {
  ttt::Act8Grad g;
  if (ttt_status_t st = act8_grad_args(desc, &g)) return st;
  if (!codes || !exps || !dy || !grad)
    return fail(TTT_ERR_INVALID_ARGUMENT, "codes, exps, dy and grad must be non-NULL");
  const size_t need = ttt::act8_weight_grad_bytes(g);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  BufferList b;
  b.in("codes", codes, (size_t)(g.rows * g.d_in));
  b.in("dy", dy, (size_t)((g.rows - 1) * g.dys + g.d_out) * ttt::dtype_bytes(g.dt));
  b.out("grad", grad, (size_t)(g.d_in * g.d_out) * ttt::dtype_bytes(g.grad_dt));
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = b.check()) return st;
  if (ttt_status_t st = b.check_against(range("exps", exps, exps_bytes(g.rows, g.d_in)))) return st;
  const hipError_t e = ttt::launch_act8_weight_grad(g, codes, exps, dy, grad, ws,
                                                    static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "act8_weight_grad");
}

}  // extern "C"
