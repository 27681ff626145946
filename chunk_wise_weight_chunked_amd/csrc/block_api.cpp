// block_api.cpp -- C ABI of the block operators (include/ttt_block.h):
// validation, workspace planning and the launch sequence on the caller's
// stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ttt_block.h"
#include "api_common.h"
#include "block.h"

using namespace ttt::api;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;

// ------------------------------------------------ residual addition + norm
ttt_status_t norm_args(const ttt_addnorm_desc_t* d, ttt::NormArgs* a) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->rows < 1) return fail(TTT_ERR_INVALID_ARGUMENT, "rows must be >= 1");
  if (d->rows > INT32_MAX) return fail(TTT_ERR_UNSUPPORTED, "rows must be < 2^31");
  if (d->d < 1) return fail(TTT_ERR_INVALID_ARGUMENT, "d must be >= 1");
  if (d->d % 8 || d->d > ttt::kNormMaxD)
    return fail(TTT_ERR_UNSUPPORTED, "d must be a multiple of 8, at most %lld",
                (long long)ttt::kNormMaxD);
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  if (d->res_dtype != d->dtype && d->res_dtype != TTT_F32)
    return fail(TTT_ERR_INVALID_ARGUMENT, "res_dtype must be dtype or TTT_F32");
  for (int64_t st : {d->x_stride, d->y_stride}) {
    if (st < d->d) return fail(TTT_ERR_INVALID_ARGUMENT, "x_stride and y_stride must be >= d");
    if (st % 8 || st > kMaxStride)
      return fail(TTT_ERR_UNSUPPORTED, "x_stride and y_stride must be multiples of 8, at most 2^40");
  }
  for (int64_t st : {d->x_stride, d->y_stride})
    if ((__int128)st * d->rows > ((__int128)1 << 56))
      return fail(TTT_ERR_UNSUPPORTED, "a tensor must span less than 2^56 values");
  if (!std::isfinite(d->eps) || d->eps < 0)
    return fail(TTT_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (d->out != TTT_NORM_SAME && d->out != TTT_NORM_FP8)
    return fail(TTT_ERR_INVALID_ARGUMENT, "out must be TTT_NORM_SAME or TTT_NORM_FP8");
  if (d->scale_group != 0 && d->scale_group != ttt::kNormScaleGroup)
    return fail(TTT_ERR_INVALID_ARGUMENT, "scale_group must be 0 or %d", ttt::kNormScaleGroup);
  if (d->scale_group && d->out != TTT_NORM_FP8)
    return fail(TTT_ERR_INVALID_ARGUMENT, "scale_group needs out = TTT_NORM_FP8");
  if (d->scale_group && d->d % ttt::kNormScaleGroup)
    return fail(TTT_ERR_UNSUPPORTED, "d must be a multiple of scale_group");
  *a = ttt::NormArgs{d->rows, d->d, d->x_stride, d->y_stride, d->eps, to_dtype(d->dtype),
                     to_dtype(d->res_dtype), d->out == TTT_NORM_FP8, d->scale_group != 0};
  return TTT_OK;
}

// Bytes from the first to behind the last element of rows `stride` apart.
size_t rows_bytes(const ttt::NormArgs& a, int64_t stride, size_t es) {
  return (size_t)((a.rows - 1) * stride + a.d) * es;
}

// ---------------------------------------------------------- linear attention
ttt_status_t linattn_dims(const ttt_linattn_desc_t* d) {
  if (!d) return fail(TTT_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->batch < 1 || d->seq_len < 1 || d->heads < 1 || d->kv_heads < 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "batch, seq_len, heads and kv_heads must be >= 1");
  if (d->heads % d->kv_heads)
    return fail(TTT_ERR_INVALID_ARGUMENT, "heads must be a multiple of kv_heads");
  // what one launch holds: its threads, up to 1024 for each head, are counted in 32 bits
  if (d->heads > 65535 || d->batch > ((int64_t)1 << 21) / d->heads)
    return fail(TTT_ERR_UNSUPPORTED, "heads must be <= 65535 and batch * heads <= 2^21");
  if (d->seq_len > ((int64_t)1 << 30) ||
      d->seq_len > ((int64_t)1 << 34) / (d->batch * d->heads))
    return fail(TTT_ERR_UNSUPPORTED, "seq_len must be <= 2^30 and batch * heads * seq_len <= 2^34");
  if (d->d_key < 1 || d->d_value < 1)
    return fail(TTT_ERR_INVALID_ARGUMENT, "d_key and d_value must be >= 1");
  if (d->d_key % 8 || d->d_value % 8 || d->d_key > ttt::kLinMaxHead || d->d_value > ttt::kLinMaxHead)
    return fail(TTT_ERR_UNSUPPORTED, "d_key and d_value must be multiples of 8, at most %d",
                ttt::kLinMaxHead);
  if (!valid_dtype(d->dtype)) return fail(TTT_ERR_INVALID_ARGUMENT, "dtype must be TTT_F32 or TTT_BF16");
  if (!std::isfinite(d->scale)) return fail(TTT_ERR_INVALID_ARGUMENT, "scale must be finite");
  for (const int64_t* st : {d->q_stride, d->k_stride, d->v_stride, d->o_stride})
    for (int i = 0; i < 3; ++i) {
      if (st[i] < 0) return fail(TTT_ERR_INVALID_ARGUMENT, "strides must be >= 0");
      if (st[i] % 8 || st[i] > kMaxStride)
        return fail(TTT_ERR_UNSUPPORTED, "strides must be multiples of 8, at most 2^40");
    }
  for (const int64_t* st : {d->q_stride, d->k_stride, d->v_stride, d->o_stride})
    if ((__int128)st[0] * (d->batch - 1) + (__int128)st[1] * (d->seq_len - 1) +
            (__int128)st[2] * (d->heads - 1) >
        ((__int128)1 << 56))
      return fail(TTT_ERR_UNSUPPORTED, "a tensor must span less than 2^56 values");
  return TTT_OK;
}

// The chunked kernels reach a chunk's rows by 32-bit offsets from its first.
constexpr int64_t kMaxTokenBytes = (int64_t)1 << 27;
ttt_status_t check_token_strides(const ttt_linattn_desc_t* d, bool with_do) {
  const int64_t es = (int64_t)ttt::dtype_bytes(to_dtype(d->dtype));
  for (const int64_t* st : {d->q_stride, d->k_stride, d->v_stride, with_do ? d->o_stride : d->q_stride})
    if (d->seq_len > 1 && st[1] * es > kMaxTokenBytes)
      return fail(TTT_ERR_UNSUPPORTED, "the token strides of q, k, v and dO must be at most 2^27 bytes");
  return TTT_OK;
}

// Whether a tensor that is written has one place for each element: every
// dimension's stride is at least the extent of those with smaller ones.
bool one_place_each(const ttt_linattn_desc_t* d, const int64_t st[3], int64_t heads, int64_t dim) {
  std::pair<int64_t, int64_t> x[3] = {{st[0], d->batch}, {st[1], d->seq_len}, {st[2], heads}};
  std::sort(x, x + 3);
  __int128 extent = dim;
  for (const auto& [stride, size] : x) {
    if (size == 1) continue;
    if (stride < extent) return false;
    extent += (__int128)stride * (size - 1);
  }
  return true;
}

size_t strided_bytes(const ttt_linattn_desc_t* d, const int64_t st[3], int64_t heads, int64_t dim) {
  return (size_t)(st[0] * (d->batch - 1) + st[1] * (d->seq_len - 1) + st[2] * (heads - 1) + dim) *
         ttt::dtype_bytes(to_dtype(d->dtype));
}

size_t state_bytes(const ttt_linattn_desc_t* d) {
  return (size_t)(d->batch * d->heads * d->d_key * d->d_value) * sizeof(float);
}

bool recurrent(const ttt_linattn_desc_t* d) { return d->seq_len <= ttt::kLinStepTokens; }

size_t forward_bytes(const ttt_linattn_desc_t* d) {
  return recurrent(d) ? 0
                      : ttt::linattn_segment_bytes(d->batch, d->heads, d->seq_len, d->d_key,
                                                   d->d_value, to_dtype(d->dtype));
}

// Backward workspace: the segments' states of dq's pass, behind them those of
// dv's where the two are made together (elsewhere dv's take the place of dq's),
// and where heads share keys and values the fp32 gradients of k and v of every
// query head.
struct BackwardPlan {
  size_t seg_bytes, dv_off, dk_off, total;
};
BackwardPlan backward_plan(const ttt_linattn_desc_t* d) {
  BackwardPlan p;
  p.seg_bytes = ttt::linattn_segment_bytes(d->batch, d->heads, d->seq_len, d->d_key, d->d_value,
                                           to_dtype(d->dtype));
  p.dv_off = align256(p.seg_bytes * (ttt::linattn_square(d->d_key, d->d_value) ? 2 : 1));
  const size_t rows = d->heads == d->kv_heads ? 0 : (size_t)(d->batch * d->heads * d->seq_len);
  p.dk_off = p.dv_off + align256(rows * d->d_value * sizeof(float));
  p.total = p.dk_off + rows * d->d_key * sizeof(float);
  return p;
}

// One token has no next one: its stride, which the limit above leaves free, must
// not reach the chunked kernels' 32-bit offsets (of 31 rows, at a last chunk's end).
ttt::LinOperand operand(const ttt_linattn_desc_t* d, const void* p, const int64_t st[3],
                        int64_t rep) {
  return {p, st[0], d->seq_len > 1 ? st[1] : 0, st[2], (int32_t)rep};
}

}  // namespace

extern "C" {

ttt_status_t ttt_addnorm_forward(const ttt_addnorm_desc_t* desc, const void* x, const void* res,
                                 const void* w, void* r, void* y, float* y_scale, void* stream) {
  ttt::NormArgs a;
  if (ttt_status_t st = norm_args(desc, &a)) return st;
  if (!x || !w || !y) return fail(TTT_ERR_INVALID_ARGUMENT, "x, w and y must be non-NULL");
  if (a.fp8 != (y_scale != nullptr))
    return fail(TTT_ERR_INVALID_ARGUMENT, "y_scale must be given for TTT_NORM_FP8 and only then");
  const size_t es = ttt::dtype_bytes(a.dt), rs = ttt::dtype_bytes(a.res_dt);
  const size_t n = (size_t)a.rows * a.d;
  BufferList b;
  b.in("x", x, rows_bytes(a, a.x_stride, es));
  b.in("res", res, n * rs);
  b.in("w", w, a.d * es);
  b.out("r", r, n * rs, res);
  b.out("y", y, rows_bytes(a, a.y_stride, a.fp8 ? 1 : es),
        !a.fp8 && a.x_stride == a.y_stride ? x : nullptr);
  b.out("y_scale", y_scale, (a.grouped ? n / ttt::kNormScaleGroup : a.rows) * sizeof(float));
  if (ttt_status_t st = b.check()) return st;
  const hipError_t e = ttt::launch_addnorm_forward(a, x, res, w, r, y, y_scale,
                                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "addnorm_forward");
}

size_t ttt_addnorm_backward_workspace_size(const ttt_addnorm_desc_t* desc) {
  ttt::NormArgs a;
  if (norm_args(desc, &a)) return 0;
  ok();
  return align256((size_t)(ttt::addnorm_backward_blocks(a) * a.d) * sizeof(float));
}

ttt_status_t ttt_addnorm_backward(const ttt_addnorm_desc_t* desc, const void* dy, const void* r,
                                  const void* w, const void* dr_out, void* dr, void* dx,
                                  float* dw, void* ws, size_t ws_bytes, void* stream) {
  ttt::NormArgs a;
  if (ttt_status_t st = norm_args(desc, &a)) return st;
  if (a.fp8) return fail(TTT_ERR_INVALID_ARGUMENT, "the backward needs out = TTT_NORM_SAME");
  if (!dy || !r || !w || !dr)
    return fail(TTT_ERR_INVALID_ARGUMENT, "dy, r, w and dr must be non-NULL");
  const size_t need =
      dw ? (size_t)(ttt::addnorm_backward_blocks(a) * a.d) * sizeof(float) : 0;
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  const size_t es = ttt::dtype_bytes(a.dt), rs = ttt::dtype_bytes(a.res_dt);
  const size_t n = (size_t)a.rows * a.d;
  BufferList b;
  b.in("dy", dy, rows_bytes(a, a.x_stride, es));
  b.in("r", r, n * rs);
  b.in("w", w, a.d * es);
  b.in("dr_out", dr_out, n * rs);
  b.out("dr", dr, n * rs, dr_out);
  b.out("dx", dx, rows_bytes(a, a.y_stride, es));
  b.out("dw", dw, a.d * sizeof(float));
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = b.check()) return st;
  const hipError_t e =
      ttt::launch_addnorm_backward(a, dy, r, w, dr_out, dr, dx, dw, static_cast<float*>(ws),
                                   static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "addnorm_backward");
}

ttt_status_t ttt_linattn_workspace_size(const ttt_linattn_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  if (ttt_status_t st = linattn_dims(desc)) return st;
  *bytes = forward_bytes(desc);
  return ok();
}

ttt_status_t ttt_linattn_backward_workspace_size(const ttt_linattn_desc_t* desc, size_t* bytes) {
  if (!bytes) return fail(TTT_ERR_INVALID_ARGUMENT, "bytes is NULL");
  if (ttt_status_t st = linattn_dims(desc)) return st;
  *bytes = backward_plan(desc).total;
  return ok();
}

ttt_status_t ttt_linattn_forward(const ttt_linattn_desc_t* desc, const void* q, const void* k,
                                 const void* v, const float* log_decay, const int32_t* lengths,
                                 const float* state_in, float* state_out, void* o, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (ttt_status_t st = linattn_dims(desc)) return st;
  if (!q || !k || !v || !log_decay || !o)
    return fail(TTT_ERR_INVALID_ARGUMENT, "q, k, v, log_decay and o must be non-NULL");
  if (!aligned(lengths, 4) || !aligned(log_decay, 4))
    return fail(TTT_ERR_INVALID_ARGUMENT, "log_decay and lengths must be 4-byte aligned");
  if (ttt_status_t st = check_token_strides(desc, false)) return st;
  if (!one_place_each(desc, desc->o_stride, desc->heads, desc->d_value))
    return fail(TTT_ERR_INVALID_ARGUMENT, "o_stride gives two elements of o one place");
  const size_t need = forward_bytes(desc);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, need)) return st;
  const int64_t H = desc->heads, G = desc->kv_heads;
  BufferList b;
  b.in("q", q, strided_bytes(desc, desc->q_stride, H, desc->d_key));
  b.in("k", k, strided_bytes(desc, desc->k_stride, G, desc->d_key));
  b.in("v", v, strided_bytes(desc, desc->v_stride, G, desc->d_value));
  b.in("state_in", state_in, state_bytes(desc));
  b.out("o", o, strided_bytes(desc, desc->o_stride, H, desc->d_value));
  b.out("state_out", state_out, state_bytes(desc), state_in);
  if (need) b.out("ws", ws, need);
  if (ttt_status_t st = b.check()) return st;
  if (ttt_status_t st = b.check_against(range("log_decay", log_decay, H * sizeof(float))))
    return st;
  if (ttt_status_t st = b.check_against(
          range("lengths", lengths, lengths ? desc->batch * sizeof(int32_t) : 0)))
    return st;
  ttt::LinArgs a{};
  a.q = operand(desc, q, desc->q_stride, 1);
  a.k = operand(desc, k, desc->k_stride, H / G);
  a.v = operand(desc, v, desc->v_stride, H / G);
  a.out = o;
  a.osb = desc->o_stride[0], a.ost = desc->o_stride[1], a.osh = desc->o_stride[2];
  a.log_decay = log_decay, a.lengths = lengths;
  a.s_in = state_in, a.s_out = state_out, a.exact_state = true;
  a.B = desc->batch, a.T = desc->seq_len, a.H = H, a.dk = desc->d_key, a.dv = desc->d_value;
  a.scale_o = a.scale_p = desc->scale, a.scale_u = 1.0f, a.late = 1;
  a.dt = to_dtype(desc->dtype);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = recurrent(desc)
                           ? ttt::launch_linattn_step(a, s)
                           : ttt::launch_linattn_chunked(a, static_cast<float*>(ws), s);
  return e == hipSuccess ? ok() : hip_fail(e, "linattn_forward");
}

ttt_status_t ttt_linattn_backward(const ttt_linattn_desc_t* desc, const void* q, const void* k,
                                  const void* v, const float* log_decay, const int32_t* lengths,
                                  const float* state_in, const void* dO, const float* dstate_out,
                                  void* dq, void* dk, void* dv, float* dstate_in, void* ws,
                                  size_t ws_bytes, void* stream) {
  if (ttt_status_t st = linattn_dims(desc)) return st;
  if (!q || !k || !v || !log_decay || !dO || !dq || !dk || !dv)
    return fail(TTT_ERR_INVALID_ARGUMENT,
                "q, k, v, log_decay, dO, dq, dk and dv must be non-NULL");
  if (!aligned(lengths, 4) || !aligned(log_decay, 4))
    return fail(TTT_ERR_INVALID_ARGUMENT, "log_decay and lengths must be 4-byte aligned");
  if (ttt_status_t st = check_token_strides(desc, true)) return st;
  const BackwardPlan plan = backward_plan(desc);
  if (ttt_status_t st = check_workspace(ws, ws_bytes, plan.total)) return st;
  const int64_t B = desc->batch, T = desc->seq_len, H = desc->heads, G = desc->kv_heads;
  const int64_t K = desc->d_key, V = desc->d_value, rep = H / G;
  const ttt::Dtype dt = to_dtype(desc->dtype);
  const size_t es = ttt::dtype_bytes(dt);
  BufferList b;
  b.in("q", q, strided_bytes(desc, desc->q_stride, H, K));
  b.in("k", k, strided_bytes(desc, desc->k_stride, G, K));
  b.in("v", v, strided_bytes(desc, desc->v_stride, G, V));
  b.in("dO", dO, strided_bytes(desc, desc->o_stride, H, V));
  b.in("state_in", state_in, state_bytes(desc));
  b.in("dstate_out", dstate_out, state_bytes(desc));
  b.out("dq", dq, (size_t)(B * T * H * K) * es);
  b.out("dk", dk, (size_t)(B * T * G * K) * es);
  b.out("dv", dv, (size_t)(B * T * G * V) * es);
  b.out("dstate_in", dstate_in, state_bytes(desc), dstate_out);
  if (plan.total) b.out("ws", ws, plan.total);
  if (ttt_status_t st = b.check()) return st;
  if (ttt_status_t st = b.check_against(range("log_decay", log_decay, H * sizeof(float))))
    return st;
  if (ttt_status_t st =
          b.check_against(range("lengths", lengths, lengths ? B * sizeof(int32_t) : 0)))
    return st;

  hipStream_t s = static_cast<hipStream_t>(stream);
  float* seg = static_cast<float*>(ws);
  const bool shared_heads = rep > 1;
  char* const wsb = static_cast<char*>(ws);
  const ttt::LinOperand oq = operand(desc, q, desc->q_stride, 1),
                        ok_ = operand(desc, k, desc->k_stride, rep),
                        ov = operand(desc, v, desc->v_stride, rep),
                        od = operand(desc, dO, desc->o_stride, 1);
  ttt::LinArgs base{};
  base.log_decay = log_decay, base.lengths = lengths;
  base.B = B, base.T = T, base.H = H, base.dt = dt;
  base.scale_p = desc->scale;

  // dq = the operator with (dO, v, k) for (q, k, v); its state is S transposed
  ttt::LinArgs aq = base;
  aq.q = od, aq.k = ov, aq.v = ok_, aq.dk = V, aq.dv = K;
  aq.out = dq, aq.osb = T * H * K, aq.ost = H * K, aq.osh = K;
  aq.s_in = state_in, aq.s_trans = true;
  aq.scale_o = desc->scale, aq.scale_u = 1.0f, aq.late = 1;

  // dk and dv run from the last token; their state starts from dstate_out and
  // ends as dstate_in, dk's being dv's transposed.  With shared heads they go to
  // the workspace per query head and are summed from there.
  struct Out {
    void* p;
    int64_t sb, st, sh;
  };
  const auto out_of = [&](void* out, size_t part_off, int64_t d) {
    return shared_heads ? Out{wsb + part_off, H * T * d, d, T * d} : Out{out, T * G * d, G * d, d};
  };
  const Out out_v = out_of(dv, plan.dv_off, V), out_k = out_of(dk, plan.dk_off, K);
  ttt::LinArgs av = base;
  av.out_f32 = shared_heads, av.s_in = dstate_out, av.scale_o = 1.0f, av.scale_u = desc->scale;
  av.late = 0, av.reverse = true;
  ttt::LinArgs ak = av;
  av.q = ok_, av.k = oq, av.v = od, av.dk = K, av.dv = V;
  av.out = out_v.p, av.osb = out_v.sb, av.ost = out_v.st, av.osh = out_v.sh;
  av.s_out = dstate_in, av.exact_state = true;
  ak.q = ov, ak.k = od, ak.v = oq, ak.dk = V, ak.dv = K;
  ak.out = out_k.p, ak.osb = out_k.sb, ak.ost = out_k.st, ak.osh = out_k.sh;
  ak.s_trans = true;

  hipError_t e = hipSuccess;
  const auto run = [&](const ttt::LinArgs& a, float* states) {
    if (e == hipSuccess) e = ttt::launch_linattn_chunked(a, states, s);
  };
  float* seg_v = seg;
  if (plan.seg_bytes && ttt::linattn_square(K, V)) {
    seg_v = seg + plan.seg_bytes / sizeof(float);
    ttt::LinArgs both[2] = {aq, av};
    both[0].exact_state = true;
    e = ttt::launch_linattn_starts(both, 2, seg, s);
    aq.seg_ready = av.seg_ready = true;
  }
  run(aq, seg);
  if (ttt::linattn_square(K, V) && dt == ttt::Dtype::BF16) {
    av.pair = true, av.w = ov;
    av.out2 = out_k.p, av.osb2 = out_k.sb, av.ost2 = out_k.st, av.osh2 = out_k.sh;
    run(av, seg_v);
  } else if (plan.seg_bytes) {
    // dk takes the segments' states that dv's pass leaves, and so reads no
    // dstate_out, which dv's pass may have replaced
    run(av, seg_v);
    ak.seg_trans = true;
    run(ak, seg_v);
  } else {
    run(ak, nullptr);  // reads dstate_out, which dv's pass may replace
    run(av, nullptr);
  }
  if (shared_heads && e == hipSuccess)
    e = ttt::launch_linattn_sum_heads(static_cast<const float*>(out_k.p), dk, K,
                                      static_cast<const float*>(out_v.p), dv, V, B, T, G, rep, dt,
                                      s);
  return e == hipSuccess ? ok() : hip_fail(e, "linattn_backward");
}

}  // extern "C"
