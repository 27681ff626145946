"""Python binding of the sequence operators (the C ABI declared in
include/ttt_seq.h): the embedding lookup and its gradient, the gated linear
recurrence with its gradients, and activations kept in 8 bits with the weight
gradient from them.

Like block, this is argument marshalling only, over the same library
(ttt_mlp.load()): the functions named as the C entry points take raw descriptors
and buffers; the others allocate outputs and workspace with torch and call them,
on the current stream of the tensors' device or on the one given as stream= (a
torch stream, or a raw handle of a stream of that device; 0 is its null stream).
The inputs' memory has to last until that stream is done with it.  There is no
fallback.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import ttt_mlp as _tm
from .block import _dtype, _on, _rows, _run, _same_device, _strided
from .ttt_mlp import _check, _ptr

GATEDREC_TILE = 128  # tokens between two states that gatedrec_forward saves
ACT8_GROUP = 32      # values of a row that share an exponent

EXPORTS = (
    "ttt_embed_forward", "ttt_embed_backward_workspace_size", "ttt_embed_backward",
    "ttt_gatedrec_saved_size", "ttt_gatedrec_workspace_size",
    "ttt_gatedrec_backward_workspace_size", "ttt_gatedrec_forward", "ttt_gatedrec_backward",
    "ttt_act8_store", "ttt_act8_load", "ttt_act8_weight_grad_workspace_size",
    "ttt_act8_weight_grad",
)

_FLOATS = (torch.bfloat16, torch.float32)


class ttt_embed_desc_t(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("id_bytes", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
    ]


class ttt_gatedrec_desc_t(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seq_len", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("x_stride", ctypes.c_int64 * 2),
        ("decay_stride", ctypes.c_int64 * 2),
        ("input_stride", ctypes.c_int64 * 2),
        ("out_stride", ctypes.c_int64 * 2),
    ]


class ttt_act8_desc_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("x_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int),
    ]


class ttt_act8_wgrad_desc_t(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("d_in", ctypes.c_int64),
        ("d_out", ctypes.c_int64),
        ("dy_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("grad_dtype", ctypes.c_int),
        ("accumulate", ctypes.c_int32),
    ]


@functools.lru_cache(maxsize=None)
def _load():
    lib = _tm.load()
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    szp = ctypes.POINTER(sz)
    ed, gd = ctypes.POINTER(ttt_embed_desc_t), ctypes.POINTER(ttt_gatedrec_desc_t)
    ad, wd = ctypes.POINTER(ttt_act8_desc_t), ctypes.POINTER(ttt_act8_wgrad_desc_t)
    for name, args in (
            ("ttt_embed_forward", [ed] + [vp] * 4),
            ("ttt_embed_backward_workspace_size", [ed, szp]),
            ("ttt_embed_backward", [ed] + [vp] * 4 + [sz, vp]),
            ("ttt_gatedrec_saved_size", [gd, szp]),
            ("ttt_gatedrec_workspace_size", [gd, szp]),
            ("ttt_gatedrec_backward_workspace_size", [gd, szp]),
            ("ttt_gatedrec_forward", [gd] + [vp] * 10 + [sz, vp]),
            ("ttt_gatedrec_backward", [gd] + [vp] * 14 + [sz, vp]),
            ("ttt_act8_store", [ad] + [vp] * 4),
            ("ttt_act8_load", [ad] + [vp] * 4),
            ("ttt_act8_weight_grad_workspace_size", [wd, szp]),
            ("ttt_act8_weight_grad", [wd] + [vp] * 5 + [sz, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i
    return lib


def _size(fn, desc) -> int:
    n = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def _bytes(ws, ws_bytes) -> int:
    if ws_bytes is None:
        return 0 if ws is None else ws.numel() * ws.element_size()
    return int(ws_bytes)


def _new_ws(need, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


# ---------------------------------------------------------------- embedding
def make_embed_desc(tokens, vocab, d, dtype, out_dtype=None, scale=1.0, id_bytes=8,
                    accumulate=False) -> ttt_embed_desc_t:
    return ttt_embed_desc_t(int(tokens), int(vocab), int(d), float(scale), _dtype(dtype),
                            _dtype(dtype if out_dtype is None else out_dtype), int(id_bytes),
                            int(accumulate))


def ttt_embed_forward(desc, ids, table, out, stream=None) -> None:
    _run(_load().ttt_embed_forward, stream, table, ctypes.byref(desc), _ptr(ids), _ptr(table),
         _ptr(out))


def ttt_embed_backward_workspace_size(desc) -> int:
    return _size(_load().ttt_embed_backward_workspace_size, desc)


def ttt_embed_backward(desc, ids, dout, grad, ws, ws_bytes=None, stream=None) -> None:
    _run(_load().ttt_embed_backward, stream, dout, ctypes.byref(desc), _ptr(ids), _ptr(dout),
         _ptr(grad), _ptr(ws), _bytes(ws, ws_bytes))


@functools.lru_cache(maxsize=256)
def _embed_plan(tokens, vocab, d, dtype, out_dtype, scale, id_bytes, accumulate, backward):
    """(descriptor, workspace bytes) of a call."""
    desc = make_embed_desc(tokens, vocab, d, dtype, out_dtype, scale, id_bytes, accumulate)
    return desc, ttt_embed_backward_workspace_size(desc) if backward else 0


def _embed_checks(ids, rows, what, out_dtype):
    if ids.dtype not in (torch.int64, torch.int32):
        raise ValueError("ids must be int64 or int32")
    if rows.dtype not in _FLOATS:
        raise ValueError(f"{what} must be bfloat16 or float32")
    if out_dtype not in (rows.dtype, torch.float32):
        raise ValueError(f"the result's type must be {what}'s or float32")
    _same_device(rows, ids)


def embed_forward(ids, table, scale=1.0, out_dtype=None, stream=None):
    """out[..., :] = scale * table[ids], zeros where an id is outside the table.

    ids int64 or int32 of any shape, table [vocab][d] bf16 or fp32, both contiguous.  Returns
    [*ids.shape][d] in the table's type, or in out_dtype=torch.float32."""
    if stream is not None:
        with _on(stream, table):
            return embed_forward(ids, table, scale, out_dtype)
    out_dtype = table.dtype if out_dtype is None else out_dtype
    _embed_checks(ids, table, "table", out_dtype)
    if table.dim() != 2 or 0 in table.shape:
        raise ValueError("table must be [vocab][d]")
    out = torch.empty((*ids.shape, table.shape[1]), dtype=out_dtype, device=table.device)
    if ids.numel():
        desc, _ = _embed_plan(ids.numel(), table.shape[0], table.shape[1], table.dtype, out_dtype,
                              float(scale), ids.element_size(), False, False)
        ttt_embed_forward(desc, ids, table, out)
    return out


def embed_backward(dout, ids, vocab, scale=1.0, grad_dtype=None, grad=None, ws=None, stream=None):
    """The table's gradient: grad[v] = scale * (the sum of dout over the tokens with id v).

    dout [*ids.shape][d] bf16 or fp32, contiguous.  Returns grad [vocab][d] in grad_dtype
    (float32 unless given; dout's type or float32).  With grad= the sums are added to that tensor,
    which is returned: rows without tokens are not touched."""
    if stream is not None:
        with _on(stream, dout):
            return embed_backward(dout, ids, vocab, scale, grad_dtype, grad, ws)
    if grad_dtype is None:
        grad_dtype = torch.float32 if grad is None else grad.dtype
    _embed_checks(ids, dout, "dout", grad_dtype)
    vocab = int(vocab)
    if dout.dim() < 1 or dout.shape[:-1] != ids.shape or dout.shape[-1] == 0:
        raise ValueError("dout must be [*ids.shape][d]")
    d = dout.shape[-1]
    if grad is not None and (grad.shape != (vocab, d) or grad.dtype != grad_dtype):
        raise ValueError(f"grad must be [{vocab}][{d}] of {grad_dtype}")
    _same_device(dout, grad, ws)
    if not ids.numel():
        return (torch.zeros((vocab, d), dtype=grad_dtype, device=dout.device) if grad is None
                else grad)
    desc, need = _embed_plan(ids.numel(), vocab, d, dout.dtype, grad_dtype, float(scale),
                             ids.element_size(), grad is not None, True)
    if grad is None:
        grad = torch.empty((vocab, d), dtype=grad_dtype, device=dout.device)
    ttt_embed_backward(desc, ids, dout, grad, _new_ws(need, dout.device) if ws is None else ws)
    return grad


# ----------------------------------------------------- gated linear recurrence
def make_gatedrec_desc(batch, seq_len, d, dtype, x_stride=None, decay_stride=None,
                       input_stride=None, out_stride=None) -> ttt_gatedrec_desc_t:
    """Strides are (batch, token) in values; None: contiguous [B][T][d]."""
    def st(given):
        return (ctypes.c_int64 * 2)(*((seq_len * d, d) if given is None else given))

    return ttt_gatedrec_desc_t(int(batch), int(seq_len), int(d), _dtype(dtype), st(x_stride),
                               st(decay_stride), st(input_stride), st(out_stride))


def ttt_gatedrec_saved_size(desc) -> int:
    return _size(_load().ttt_gatedrec_saved_size, desc)


def ttt_gatedrec_workspace_size(desc) -> int:
    return _size(_load().ttt_gatedrec_workspace_size, desc)


def ttt_gatedrec_backward_workspace_size(desc) -> int:
    return _size(_load().ttt_gatedrec_backward_workspace_size, desc)


def ttt_gatedrec_forward(desc, x, decay_gate, input_gate, rate, lengths, state_in, state_out, h,
                         saved=None, ws=None, ws_bytes=None, stream=None) -> None:
    _run(_load().ttt_gatedrec_forward, stream, x, ctypes.byref(desc), _strided(x),
         _strided(decay_gate), _strided(input_gate), _ptr(rate), _ptr(lengths), _ptr(state_in),
         _ptr(state_out), _strided(h), _ptr(saved), _ptr(ws), _bytes(ws, ws_bytes))


def ttt_gatedrec_backward(desc, x, decay_gate, input_gate, rate, lengths, saved, dh, dstate_out,
                          dx, ddecay, dinput, drate, dstate_in, ws=None, ws_bytes=None,
                          stream=None) -> None:
    _run(_load().ttt_gatedrec_backward, stream, x, ctypes.byref(desc), _strided(x),
         _strided(decay_gate), _strided(input_gate), _ptr(rate), _ptr(lengths), _ptr(saved),
         _strided(dh), _ptr(dstate_out), _ptr(dx), _ptr(ddecay), _ptr(dinput), _ptr(drate),
         _ptr(dstate_in), _ptr(ws), _bytes(ws, ws_bytes))


@functools.lru_cache(maxsize=256)
def _gatedrec_plan(shape, xs, gs, ins, os, dtype, backward):
    """(descriptor, workspace bytes) of a call's shape and strides."""
    for s in (xs, gs, ins) + (() if os is None else (os,)):
        if s[2] != 1 and shape[2] > 1:
            raise ValueError("the last dimension must be contiguous")
    # a dimension of one element has no stride to speak of (torch may give any)
    real = lambda st: [0 if n == 1 else x for n, x in zip(shape, st[:2])]  # noqa: E731
    desc = make_gatedrec_desc(*shape, dtype, real(xs), real(gs), real(ins),
                              None if os is None else real(os))
    return desc, (ttt_gatedrec_backward_workspace_size if backward
                  else ttt_gatedrec_workspace_size)(desc)


def _gatedrec_checks(x, decay_gate, input_gate, rate, lengths, ws, *states):
    """What the plan does not look at: shapes, types, devices, and the fp32 tensors."""
    if x.dim() != 3 or 0 in x.shape:
        raise ValueError("x must be [B][T][d]")
    if x.dtype not in _FLOATS:
        raise ValueError("x must be bfloat16 or float32")
    for t in (decay_gate, input_gate):
        if t.shape != x.shape or t.dtype != x.dtype:
            raise ValueError("the gates must have x's shape and type")
    B, _, d = x.shape
    if rate.shape != (d,) or rate.dtype != torch.float32:
        raise ValueError(f"rate must be [{d}] float32")
    if lengths is not None and (lengths.shape != (B,) or lengths.dtype != torch.int32):
        raise ValueError(f"lengths must be [{B}] int32")
    for s in states:
        if s is not None and (s.shape != (B, d) or s.dtype != torch.float32):
            raise ValueError(f"states must be [{B}][{d}] float32")
    _same_device(x, decay_gate, input_gate, rate, lengths, ws, *states)


def gatedrec_forward(x, decay_gate, input_gate, rate, state=None, state_out=None, lengths=None,
                     save=False, ws=None, stream=None):
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(input_gate_t) x_t for each channel, with
    a_t = exp(-rate sigmoid(decay_gate_t)).

    x and the gates [B][T][d] (bf16 or fp32; any strides in multiples of 8 with a contiguous last
    dimension), rate [d] fp32 >= 0, state [B][d] fp32 or None (zeros), lengths [B] int32 or None.
    Returns (h [B][T][d], the state behind the last token, what gatedrec_backward needs with
    save=True or None); pass state_out=state to update a session's state in place."""
    if stream is not None:
        with _on(stream, x):
            return gatedrec_forward(x, decay_gate, input_gate, rate, state, state_out, lengths,
                                    save, ws)
    _gatedrec_checks(x, decay_gate, input_gate, rate, lengths, ws, state, state_out)
    desc, need = _gatedrec_plan(x.shape, x.stride(), decay_gate.stride(), input_gate.stride(),
                                None, x.dtype, False)
    B, T, d = x.shape
    h = torch.empty_like(x, memory_format=torch.contiguous_format)
    if state_out is None:
        state_out = torch.empty((B, d), dtype=torch.float32, device=x.device)
    saved = torch.empty((B, -(-T // GATEDREC_TILE), d), dtype=torch.float32,
                        device=x.device) if save else None
    ttt_gatedrec_forward(desc, x, decay_gate, input_gate, rate, lengths, state, state_out, h,
                         saved, _new_ws(need, x.device) if ws is None else ws)
    return h, state_out, saved


def gatedrec_backward(x, decay_gate, input_gate, rate, dh, saved, dstate_out=None, lengths=None,
                      ws=None, stream=None) -> dict:
    """Gradients of <dh, h> + <dstate_out, final state> for gatedrec_forward of the same arguments,
    whose third result is `saved`.  Returns a dict: x, decay_gate, input_gate (x's shape and type,
    contiguous), rate [d] and state [B][d] (fp32)."""
    if stream is not None:
        with _on(stream, x):
            return gatedrec_backward(x, decay_gate, input_gate, rate, dh, saved, dstate_out,
                                     lengths, ws)
    _gatedrec_checks(x, decay_gate, input_gate, rate, lengths, ws, dstate_out)
    B, T, d = x.shape
    if dh.shape != x.shape or dh.dtype != x.dtype:
        raise ValueError("dh must have x's shape and type")
    tiles = -(-T // GATEDREC_TILE)
    if saved is None or saved.shape != (B, tiles, d) or saved.dtype != torch.float32:
        raise ValueError(f"saved must be the forward's, [{B}][{tiles}][{d}] float32")
    _same_device(x, dh, saved)
    desc, need = _gatedrec_plan(x.shape, x.stride(), decay_gate.stride(), input_gate.stride(),
                                dh.stride(), x.dtype, True)
    new = lambda: torch.empty_like(x, memory_format=torch.contiguous_format)  # noqa: E731
    g = {"x": new(), "decay_gate": new(), "input_gate": new(),
         "rate": torch.empty(d, dtype=torch.float32, device=x.device),
         "state": torch.empty((B, d), dtype=torch.float32, device=x.device)}
    ttt_gatedrec_backward(desc, x, decay_gate, input_gate, rate, lengths, saved, dh, dstate_out,
                          g["x"], g["decay_gate"], g["input_gate"], g["rate"], g["state"],
                          _new_ws(need, x.device) if ws is None else ws)
    return g


# ---------------------------------------------------------- activations in 8 bits
def make_act8_desc(rows, d, dtype, x_stride=None) -> ttt_act8_desc_t:
    return ttt_act8_desc_t(int(rows), int(d), int(d if x_stride is None else x_stride),
                           _dtype(dtype))


def make_act8_wgrad_desc(rows, d_in, d_out, dtype, grad_dtype=torch.float32, dy_stride=None,
                         accumulate=False) -> ttt_act8_wgrad_desc_t:
    return ttt_act8_wgrad_desc_t(int(rows), int(d_in), int(d_out),
                                 int(d_out if dy_stride is None else dy_stride), _dtype(dtype),
                                 _dtype(grad_dtype), int(accumulate))


def ttt_act8_store(desc, x, codes, exps, stream=None) -> None:
    _run(_load().ttt_act8_store, stream, x, ctypes.byref(desc), _strided(x), _ptr(codes),
         _ptr(exps))


def ttt_act8_load(desc, codes, exps, x, stream=None) -> None:
    _run(_load().ttt_act8_load, stream, codes, ctypes.byref(desc), _ptr(codes), _ptr(exps),
         _strided(x))


def ttt_act8_weight_grad_workspace_size(desc) -> int:
    return _size(_load().ttt_act8_weight_grad_workspace_size, desc)


def ttt_act8_weight_grad(desc, codes, exps, dy, grad, ws=None, ws_bytes=None,
                         stream=None) -> None:
    _run(_load().ttt_act8_weight_grad, stream, codes, ctypes.byref(desc), _ptr(codes), _ptr(exps),
         _strided(dy), _ptr(grad), _ptr(ws), _bytes(ws, ws_bytes))


@functools.lru_cache(maxsize=256)
def _act8_plan(rows, d, dtype, x_stride):
    return make_act8_desc(rows, d, dtype, x_stride)


@functools.lru_cache(maxsize=256)
def _wgrad_plan(rows, d_in, d_out, dtype, grad_dtype, dy_stride, accumulate):
    desc = make_act8_wgrad_desc(rows, d_in, d_out, dtype, grad_dtype, dy_stride, accumulate)
    return desc, ttt_act8_weight_grad_workspace_size(desc)


def _act8_checks(codes, exps):
    if codes.dtype != torch.int8 or codes.dim() < 1 or 0 in codes.shape:
        raise ValueError("codes must be int8 rows")
    want = (*codes.shape[:-1], -(-codes.shape[-1] // ACT8_GROUP))
    if exps.dtype != torch.uint8 or exps.shape != want:
        raise ValueError(f"exps must be {list(want)} uint8")
    _same_device(codes, exps)


def act8_store(x, stream=None):
    """x in 8 bits: codes, int8 of x's shape, and exps, uint8 with one value for each 32 of a row:
    codes * 2^(exps - 127), the scale the smallest power of two that takes the largest of the 32 to
    at most 127 (between 2^-126 and 2^121).  A group with an infinity or a NaN stands for NaN.

    x [..., d] bf16 or fp32 (contiguous, or 2-dimensional with rows a multiple of 8 values apart;
    16-byte aligned)."""
    if stream is not None:
        with _on(stream, x):
            return act8_store(x)
    if x.dtype not in _FLOATS or x.dim() < 1 or 0 in x.shape:
        raise ValueError("x must be bfloat16 or float32 rows")
    rows, d, xs = _rows(x)
    desc = _act8_plan(rows, d, x.dtype, d if rows == 1 else xs)
    codes = torch.empty_like(x, dtype=torch.int8, memory_format=torch.contiguous_format)
    exps = torch.empty((*x.shape[:-1], -(-d // ACT8_GROUP)), dtype=torch.uint8, device=x.device)
    ttt_act8_store(desc, x, codes, exps)
    return codes, exps


def act8_load(codes, exps, dtype=torch.bfloat16, stream=None):
    """The values that act8_store's results stand for, exactly, in bf16 or fp32."""
    if stream is not None:
        with _on(stream, codes):
            return act8_load(codes, exps, dtype)
    _act8_checks(codes, exps)
    if dtype not in _FLOATS:
        raise ValueError("dtype must be bfloat16 or float32")
    d = codes.shape[-1]
    x = torch.empty_like(codes, dtype=dtype)
    ttt_act8_load(_act8_plan(codes.numel() // d, d, dtype, d), codes, exps, x)
    return x


def act8_weight_grad(codes, exps, dy, grad_dtype=torch.float32, grad=None, ws=None, stream=None):
    """The gradient x^T dy [d_in][d_out] of a weight, with x [..., d_in] as act8_store kept it and
    dy [..., d_out] bf16 or fp32 (contiguous, or 2-dimensional with rows a multiple of 8 values
    apart), in grad_dtype (float32, or dy's type).  With grad= (float32) it is added to that tensor,
    which is returned."""
    if stream is not None:
        with _on(stream, codes):
            return act8_weight_grad(codes, exps, dy, grad_dtype, grad, ws)
    _act8_checks(codes, exps)
    if dy.dtype not in _FLOATS or dy.shape[:-1] != codes.shape[:-1] or 0 in dy.shape:
        raise ValueError("dy must be bfloat16 or float32 with the codes' rows")
    if grad_dtype not in (dy.dtype, torch.float32):
        raise ValueError("grad_dtype must be float32 or dy's type")
    rows, m, dys = _rows(dy)
    d = codes.shape[-1]
    if grad is not None and (grad.shape != (d, m) or grad.dtype != torch.float32
                             or grad_dtype != torch.float32):
        raise ValueError(f"grad must be [{d}][{m}] float32")
    _same_device(codes, dy, grad, ws)
    desc, need = _wgrad_plan(rows, d, m, dy.dtype, grad_dtype, m if rows == 1 else dys,
                             grad is not None)
    if grad is None:
        grad = torch.empty((d, m), dtype=grad_dtype, device=codes.device)
    ttt_act8_weight_grad(desc, codes, exps, dy, grad,
                         _new_ws(need, codes.device) if ws is None else ws)
    return grad
