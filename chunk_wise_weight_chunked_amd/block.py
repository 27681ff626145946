"""Python binding of the block operators (the C ABI declared in
include/ttt_block.h): the residual addition with the root-mean-square norm, and
linear attention with a decay for each head, each with its gradients.

Like ttt_mlp, this is argument marshalling only, over the same library
(ttt_mlp.load()): the functions named as the C entry points take raw
descriptors and buffers; add_rmsnorm, add_rmsnorm_backward, linattn_forward
and linattn_backward allocate outputs and workspace with torch and call them, on
the current stream of the tensors' device or on the one given as stream= (a torch
stream, or a raw handle of a stream of that device; 0 is its null stream).  The
inputs' memory has to last until that stream is done with it.  There is no fallback.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import ttt_mlp as _tm
from .ttt_mlp import TTT_BF16, TTT_F32, TTTError, _check, _ptr, _stream, ttt_last_error

TTT_NORM_SAME, TTT_NORM_FP8 = 0, 1
NORM_EPS = 1e-6

EXPORTS = (
    "ttt_addnorm_forward", "ttt_addnorm_backward_workspace_size", "ttt_addnorm_backward",
    "ttt_linattn_workspace_size", "ttt_linattn_backward_workspace_size", "ttt_linattn_forward",
    "ttt_linattn_backward",
)

_DTYPES = {torch.float32: TTT_F32, torch.bfloat16: TTT_BF16}


class ttt_addnorm_desc_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("dtype", ctypes.c_int),
        ("res_dtype", ctypes.c_int),
        ("out", ctypes.c_int),
        ("scale_group", ctypes.c_int32),
    ]


class ttt_linattn_desc_t(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seq_len", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("kv_heads", ctypes.c_int64),
        ("d_key", ctypes.c_int64),
        ("d_value", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("q_stride", ctypes.c_int64 * 3),
        ("k_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3),
        ("o_stride", ctypes.c_int64 * 3),
    ]


@functools.lru_cache(maxsize=None)
def _load():
    lib = _tm.load()
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    nd, ld = ctypes.POINTER(ttt_addnorm_desc_t), ctypes.POINTER(ttt_linattn_desc_t)
    szp = ctypes.POINTER(sz)
    for name, args, res in (
            ("ttt_addnorm_forward", [nd] + [vp] * 7, ctypes.c_int),
            ("ttt_addnorm_backward_workspace_size", [nd], sz),
            ("ttt_addnorm_backward", [nd] + [vp] * 8 + [sz, vp], ctypes.c_int),
            ("ttt_linattn_workspace_size", [ld, szp], ctypes.c_int),
            ("ttt_linattn_backward_workspace_size", [ld, szp], ctypes.c_int),
            ("ttt_linattn_forward", [ld] + [vp] * 9 + [sz, vp], ctypes.c_int),
            ("ttt_linattn_backward", [ld] + [vp] * 13 + [sz, vp], ctypes.c_int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    return lib


def _dtype(t) -> int:
    return _DTYPES[t] if isinstance(t, torch.dtype) else int(t)


def _strided(t):
    """Address of a device tensor whose strides are passed beside it."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must be device (cuda) tensors")
    return t.data_ptr()


def _run(fn, stream, like, *args):
    """fn(*args, stream): the stream given, or the current one of the device of `like`.  A null
    handle is the null stream of the device that is current, so that device is made current."""
    if stream is None and getattr(like, "is_cuda", False):
        where = like.get_device()
        handle = torch._C._cuda_getCurrentRawStream(where)
    else:
        where = stream.device.index if isinstance(stream, torch.cuda.Stream) else None
        handle = _stream(stream)
    if where is None or where == torch._C._cuda_getDevice():
        return _check(fn(*args, handle))
    with torch.cuda.device(where):
        return _check(fn(*args, handle))


def _on(stream, like):
    """A tensor-level call with stream=s allocates on s as well: its outputs and its workspace
    are that stream's, so no other stream's allocation can take their memory while s still
    works on it.  A raw handle is a stream of the device of `like`."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        # ExternalStream takes a null pointer as none given and makes a stream of its own
        stream = (torch.cuda.ExternalStream(handle, device=like.device) if handle
                  else torch.cuda.default_stream(like.device))
    return torch.cuda.stream(stream)


# ------------------------------------------------ residual addition and norm
def make_addnorm_desc(rows, d, dtype, res_dtype=None, x_stride=None, y_stride=None, eps=NORM_EPS,
                      out=TTT_NORM_SAME, scale_group=0) -> ttt_addnorm_desc_t:
    return ttt_addnorm_desc_t(int(rows), int(d), int(d if x_stride is None else x_stride),
                              int(d if y_stride is None else y_stride), float(eps), _dtype(dtype),
                              _dtype(dtype if res_dtype is None else res_dtype), int(out),
                              int(scale_group))


def ttt_addnorm_forward(desc, x, res, w, r, y, y_scale=None, stream=None) -> None:
    _run(_load().ttt_addnorm_forward, stream, x, ctypes.byref(desc), _strided(x), _ptr(res),
         _ptr(w), _ptr(r), _strided(y), _ptr(y_scale))


def ttt_addnorm_backward_workspace_size(desc) -> int:
    n = _load().ttt_addnorm_backward_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise TTTError(_tm.TTT_ERR_INVALID_ARGUMENT, ttt_last_error())
    return int(n)


def ttt_addnorm_backward(desc, dy, r, w, dr_out, dr, dx, dw, ws=None, ws_bytes=None,
                         stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _run(_load().ttt_addnorm_backward, stream, dy, ctypes.byref(desc), _strided(dy), _ptr(r),
         _ptr(w), _ptr(dr_out), _ptr(dr), _strided(dx), _ptr(dw), _ptr(ws), int(ws_bytes))


@functools.lru_cache(maxsize=256)
def _norm_plan(rows, d, x_stride, dtype, res_dtype, eps, fp8, scale_group):
    return make_addnorm_desc(rows, d, dtype, res_dtype, x_stride, d, eps,
                             TTT_NORM_FP8 if fp8 else TTT_NORM_SAME, scale_group)


def _rows(t):
    """(rows, d, values between rows) of a tensor of rows; the rows may be apart."""
    d = t.shape[-1]
    if d == 0:
        raise ValueError("the rows have no values")
    if t.stride(-1) != 1 and d > 1:
        raise ValueError("the last dimension must be contiguous")
    if t.is_contiguous():
        return t.numel() // d, d, d
    if t.dim() != 2:
        raise ValueError("rows that are apart need a 2-dimensional tensor")
    return t.shape[0], d, t.stride(0)


def _same_device(like, *tensors):
    where = like.get_device()
    for t in tensors:
        if t is not None and t.get_device() != where:
            raise ValueError(f"tensors on {like.device} and on {t.device}")


def _norm_checks(x, res, w, what):
    if x.dtype not in _DTYPES:
        raise ValueError(f"{what} must be bfloat16 or float32")
    if w.shape != x.shape[-1:] or w.dtype != x.dtype:
        raise ValueError(f"weight must be [{x.shape[-1]}] of {x.dtype}")
    if res is not None and (res.shape != x.shape or res.dtype not in (x.dtype, torch.float32)):
        raise ValueError(f"the residual must have {what}'s shape and its type or float32")


def add_rmsnorm(x, res, weight, eps=NORM_EPS, out_dtype=None, scale_group=0, r_out=None,
                stream=None):
    """r = x + res, y = r / sqrt(mean(r^2) + eps) * weight over the last dimension.

    x [..., d] bf16 or fp32 (contiguous, or 2-dimensional with rows a multiple of 8 values apart;
    16-byte aligned), weight [d] of its type, res (or None) of its type or fp32.  Returns
    (y, r, scale).  r has res's type (written to r_out if given, which may be res itself; None
    without a residual); y has x's
    type and scale is None, or with out_dtype=torch.float8_e4m3fn y is 8-bit and scale holds one
    fp32 value for each row, or for each 128 values of a row (scale_group=128): y * scale is the
    norm."""
    if stream is not None:
        with _on(stream, x):
            return add_rmsnorm(x, res, weight, eps, out_dtype, scale_group, r_out)
    _norm_checks(x, res, weight, "x")
    _same_device(x, res, weight, r_out)
    fp8 = out_dtype is torch.float8_e4m3fn
    if not fp8 and out_dtype not in (None, x.dtype):
        raise ValueError("out_dtype must be None, x's type or float8_e4m3fn")
    if r_out is not None and (res is None or r_out.shape != res.shape or r_out.dtype != res.dtype):
        raise ValueError("r_out needs a residual and its shape and type")
    rows, d, xs = _rows(x)
    if rows == 0:
        raise ValueError("x has no rows")
    desc = _norm_plan(rows, d, xs, x.dtype, x.dtype if res is None else res.dtype, float(eps),
                      fp8, int(scale_group))
    # contiguous outputs, whatever the rows of x are apart
    y = (torch.empty(x.shape, dtype=out_dtype, device=x.device) if fp8
         else torch.empty_like(x, memory_format=torch.contiguous_format))
    r = (None if res is None
         else torch.empty_like(res, memory_format=torch.contiguous_format) if r_out is None
         else r_out)
    scale = None
    if fp8:
        shape = x.shape[:-1] + (d // scale_group if scale_group else 1,)
        scale = torch.empty(shape, dtype=torch.float32, device=x.device)
    ttt_addnorm_forward(desc, x, res, weight, r, y, scale)
    return y, r, scale


def add_rmsnorm_backward(dy, r, weight, eps=NORM_EPS, dr=None, stream=None):
    """Gradients of <dy, y> + <dr, r> for y = norm(r) * weight: r is add_rmsnorm's (x itself where
    it had no residual), dr the gradient that reaches r from its other uses, or None.  Returns
    (dr, dx, dweight): the gradient of the sum in r's type, the same in dy's type (the same
    tensor where the types are equal), and the fp32 gradient of the weight."""
    if stream is not None:
        with _on(stream, dy):
            return add_rmsnorm_backward(dy, r, weight, eps, dr)
    _norm_checks(dy, r, weight, "dy")
    _same_device(dy, r, weight, dr)
    if dr is not None and (dr.shape != r.shape or dr.dtype != r.dtype):
        raise ValueError("dr must have r's shape and type")
    rows, d, xs = _rows(dy)
    if rows == 0:
        raise ValueError("dy has no rows")
    desc = _norm_plan(rows, d, xs, dy.dtype, r.dtype, float(eps), False, 0)
    out = torch.empty(r.shape, dtype=r.dtype, device=r.device)
    dx = None if r.dtype == dy.dtype else torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    dw = torch.empty(d, dtype=torch.float32, device=dy.device)
    ws = torch.empty(ttt_addnorm_backward_workspace_size(desc), dtype=torch.uint8,
                     device=dy.device)
    ttt_addnorm_backward(desc, dy, r, weight, dr, out, dx, dw, ws)
    return out, out if dx is None else dx, dw


# ---------------------------------------------------------- linear attention
def make_linattn_desc(batch, seq_len, heads, kv_heads, d_key, d_value, dtype, scale,
                      q_stride=None, k_stride=None, v_stride=None,
                      o_stride=None) -> ttt_linattn_desc_t:
    """Strides are (batch, token, head) in values; None: contiguous [B][T][heads][d]."""
    def st(given, n, d):
        return (ctypes.c_int64 * 3)(*((seq_len * n * d, n * d, d) if given is None else given))

    return ttt_linattn_desc_t(int(batch), int(seq_len), int(heads), int(kv_heads), int(d_key),
                              int(d_value), _dtype(dtype), float(scale),
                              st(q_stride, heads, d_key), st(k_stride, kv_heads, d_key),
                              st(v_stride, kv_heads, d_value), st(o_stride, heads, d_value))


def _size(fn, desc) -> int:
    n = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ttt_linattn_workspace_size(desc) -> int:
    return _size(_load().ttt_linattn_workspace_size, desc)


def ttt_linattn_backward_workspace_size(desc) -> int:
    return _size(_load().ttt_linattn_backward_workspace_size, desc)


def ttt_linattn_forward(desc, q, k, v, log_decay, lengths, state_in, state_out, o, ws=None,
                        ws_bytes=None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _run(_load().ttt_linattn_forward, stream, q, ctypes.byref(desc), _strided(q), _strided(k),
         _strided(v), _ptr(log_decay), _ptr(lengths), _ptr(state_in), _ptr(state_out), _strided(o),
         _ptr(ws), int(ws_bytes))


def ttt_linattn_backward(desc, q, k, v, log_decay, lengths, state_in, dO, dstate_out, dq, dk, dv,
                         dstate_in, ws=None, ws_bytes=None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _run(_load().ttt_linattn_backward, stream, q, ctypes.byref(desc), _strided(q), _strided(k),
         _strided(v), _ptr(log_decay), _ptr(lengths), _ptr(state_in), _strided(dO),
         _ptr(dstate_out), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dstate_in), _ptr(ws), int(ws_bytes))


def _value(scale):
    """A scale as the plans are kept by: its value, never the object given."""
    return None if scale is None else float(scale)


@functools.lru_cache(maxsize=256)
def _linattn_plan(q, qs, k, ks, v, vs, os, dtype, scale, backward):
    """(descriptor, workspace bytes) of a call's shapes and strides."""
    if len(q) != 4 or len(k) != 4 or len(v) != 4:
        raise ValueError("q, k and v must be [B][T][heads][d]")
    if k[:2] != q[:2] or v[:3] != k[:3] or k[3] != q[3]:
        raise ValueError(f"shapes do not match: q {tuple(q)}, k {tuple(k)}, v {tuple(v)}")
    if qs[3] != 1 or ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last dimension must be contiguous")
    if dtype not in _DTYPES:
        raise ValueError("q, k and v must be of one type, bfloat16 or float32")
    # a dimension of one element has no stride to speak of (torch may give any)
    real = lambda shape, st: [0 if n == 1 else x for n, x in zip(shape, st[:3])]  # noqa: E731
    desc = make_linattn_desc(q[0], q[1], q[2], k[2], q[3], v[3], dtype,
                             q[3] ** -0.5 if scale is None else scale, real(q, qs), real(k, ks),
                             real(v, vs), None if os is None else real(q, os))
    size = ttt_linattn_backward_workspace_size if backward else ttt_linattn_workspace_size
    return desc, size(desc)


def _linattn_checks(q, k, v, log_decay, lengths, ws, *states):
    """What the plan does not look at: types, devices, and the small and the fp32 tensors."""
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must be of one type, bfloat16 or float32")
    B, H = q.shape[0], q.shape[2]
    if log_decay.shape != (H,) or log_decay.dtype != torch.float32:
        raise ValueError(f"log_decay must be [{H}] float32")
    if lengths is not None and (lengths.shape != (B,) or lengths.dtype != torch.int32):
        raise ValueError(f"lengths must be [{B}] int32")
    for s in states:
        if s is not None and (s.shape != (B, H, q.shape[3], v.shape[3])
                              or s.dtype != torch.float32):
            raise ValueError(f"states must be [{B}][{H}][{q.shape[3]}][{v.shape[3]}] float32")
    _same_device(q, k, v, log_decay, lengths, ws, *states)


def linattn_forward(q, k, v, log_decay, scale=None, state=None, state_out=None, lengths=None,
                    ws=None, stream=None):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t for each head.

    q [B][T][H][dk], k [B][T][G][dk], v [B][T][G][dv] (bf16 or fp32; any strides in multiples
    of 8 with a contiguous last dimension; H a multiple of G), log_decay [H] fp32, state
    [B][H][dk][dv] fp32 or None (zeros), lengths [B] int32 or None.  scale: dk^-0.5 unless
    given.  Returns (o [B][T][H][dv], the state behind the last token); pass
    state_out=state to update a session's state in place."""
    if stream is not None:
        with _on(stream, q):
            return linattn_forward(q, k, v, log_decay, scale, state, state_out, lengths, ws)
    desc, need = _linattn_plan(q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(),
                               None, q.dtype, _value(scale), False)
    _linattn_checks(q, k, v, log_decay, lengths, ws, state, state_out)
    B, T, H, dk = q.shape
    dv = v.shape[3]
    o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ttt_linattn_forward(desc, q, k, v, log_decay, lengths, state, state_out, o, ws)
    return o, state_out


def linattn_backward(q, k, v, log_decay, dO, scale=None, state=None, dstate_out=None,
                     lengths=None, ws=None, stream=None) -> dict:
    """Gradients of <dO, o> + <dstate_out, final state> for linattn_forward from `state`.
    Returns a dict: q, k, v (their shapes, contiguous) and state (fp32; None when no state was
    given)."""
    if stream is not None:
        with _on(stream, q):
            return linattn_backward(q, k, v, log_decay, dO, scale, state, dstate_out, lengths, ws)
    desc, need = _linattn_plan(q.shape, q.stride(), k.shape, k.stride(), v.shape, v.stride(),
                               dO.stride(), q.dtype, _value(scale), True)
    _linattn_checks(q, k, v, log_decay, lengths, ws, state, dstate_out)
    want = (*q.shape[:3], v.shape[3])
    if dO.shape != want or dO.dtype != q.dtype or dO.stride(3) != 1:
        raise ValueError(f"dO must be {want} of {q.dtype}, last dimension contiguous")
    _same_device(q, dO)
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    g = {"q": new(q), "k": new(k), "v": new(v), "state": None if state is None else new(state)}
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    ttt_linattn_backward(desc, q, k, v, log_decay, lengths, state, dO, dstate_out, g["q"], g["k"],
                         g["v"], g["state"], ws)
    return g
