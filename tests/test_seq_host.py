"""Host-side checks of the sequence operators' C ABI (no GPU needed): exports, and
every refusal with its documented status before the device is touched.  Invalid
calls use fake (never dereferenced) device addresses.  The 64-bit forms that the
GPU tests compare with are checked here against differences."""
import contextlib
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from chunk_wise_weight_chunked_amd import build as hipbuild
from chunk_wise_weight_chunked_amd import seq
from chunk_wise_weight_chunked_amd import ttt_mlp as tm

import _seq_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "ttt_seq.h")
A = 1 << 40  # fake addresses, 1 GiB apart
INVALID, UNSUPPORTED = tm.TTT_ERR_INVALID_ARGUMENT, tm.TTT_ERR_UNSUPPORTED
SMALL = tm.TTT_ERR_WORKSPACE_TOO_SMALL


def at(i):
    return A + (i << 30)


def refused(call, status, word):
    with pytest.raises(tm.TTTError) as e:
        call()
    assert e.value.status == status, e.value
    assert word in str(e.value), str(e.value)


def test_exports_every_declared_symbol():
    lib = seq._load()
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ttt_[a-z_0-9]+)\s*\(", text)))
    assert set(names) == set(seq.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


# ---------------------------------------------------------------- embedding
def embed_desc(**kw):
    return seq.make_embed_desc(**(dict(tokens=100, vocab=50, d=64, dtype=torch.bfloat16) | kw))


BAD_EMBED = [
    (dict(tokens=0), INVALID, "tokens"),
    (dict(vocab=0), INVALID, "vocab"),
    (dict(tokens=(1 << 28) + 1), UNSUPPORTED, "tokens"),
    (dict(vocab=(1 << 31) - 1), UNSUPPORTED, "vocab"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=60), UNSUPPORTED, "d must"),
    (dict(d=(1 << 20) + 8), UNSUPPORTED, "d must"),
    (dict(tokens=1 << 28, d=2048), UNSUPPORTED, "tokens * d"),
    (dict(vocab=1 << 30, d=2048), UNSUPPORTED, "vocab * d"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(dtype=7, out_dtype=7), INVALID, "dtype"),
    (dict(dtype=torch.float32, out_dtype=torch.bfloat16), INVALID, "out_dtype"),
    (dict(id_bytes=2), INVALID, "id_bytes"),
    (dict(accumulate=2), INVALID, "accumulate"),
]


@pytest.mark.parametrize("kw,status,word", BAD_EMBED)
def test_embed_refuses_descriptors(kw, status, word):
    d = embed_desc(**kw)
    refused(lambda: seq.ttt_embed_forward(d, at(1), at(2), at(3), 0), status, word)
    refused(lambda: seq.ttt_embed_backward_workspace_size(d), status, word)
    refused(lambda: seq.ttt_embed_backward(d, at(1), at(2), at(3), at(4), 1 << 29, 0), status, word)


def test_embed_refuses_buffers():
    d = embed_desc()
    fwd = lambda *a: (lambda: seq.ttt_embed_forward(d, *a, stream=0))  # noqa: E731
    for i in range(3):
        bad = [at(1), at(2), at(3)]
        bad[i] = None
        refused(fwd(*bad), INVALID, "non-NULL")
    refused(fwd(at(1) + 4, at(2), at(3)), INVALID, "8-byte")
    refused(fwd(at(1), at(2) + 8, at(3)), INVALID, "16-byte")
    refused(fwd(at(1), at(2), at(2) + 16), INVALID, "out overlaps table")
    refused(fwd(at(3), at(2), at(3)), INVALID, "out overlaps ids")
    narrow = embed_desc(id_bytes=4)
    refused(lambda: seq.ttt_embed_forward(narrow, at(1) + 2, at(2), at(3), 0), INVALID, "4-byte")
    need = seq.ttt_embed_backward_workspace_size(d)
    bwd = lambda *a, n=need: (lambda: seq.ttt_embed_backward(d, *a, n, 0))  # noqa: E731
    for i in range(3):
        bad = [at(1), at(2), at(3), at(4)]
        bad[i] = None
        refused(bwd(*bad), INVALID, "non-NULL")
    refused(bwd(at(1), at(2), at(3), None), INVALID, "ws is NULL")
    refused(bwd(at(1), at(2), at(3), at(4) + 64), INVALID, "256-byte")
    refused(bwd(at(1), at(2), at(3), at(4), n=need - 1), SMALL, "needed")
    refused(bwd(at(1), at(2), at(2), at(4)), INVALID, "grad overlaps dout")
    refused(bwd(at(1), at(2), at(3), at(3)), INVALID, "overlaps")
    refused(bwd(at(4), at(2), at(3), at(4)), INVALID, "ws overlaps ids")


# ----------------------------------------------------- gated linear recurrence
def rec_desc(**kw):
    return seq.make_gatedrec_desc(**(dict(batch=2, seq_len=300, d=64, dtype=torch.bfloat16) | kw))


BAD_REC = [
    (dict(batch=0), INVALID, "batch"),
    (dict(seq_len=0), INVALID, "seq_len"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=12), UNSUPPORTED, "d must"),
    (dict(d=1 << 21), UNSUPPORTED, "d must"),
    (dict(batch=(1 << 20) + 1, seq_len=1, d=8), UNSUPPORTED, "2^20"),
    (dict(batch=1, seq_len=(1 << 29) + 1, d=8), UNSUPPORTED, "2^29"),
    (dict(batch=1 << 14, seq_len=1, d=(1 << 14) + 8), UNSUPPORTED, "2^28"),
    (dict(batch=1, seq_len=1 << 26, d=1024), UNSUPPORTED, "2^35"),
    (dict(batch=1, seq_len=(1 << 62), d=8), UNSUPPORTED, "2^29"),
    (dict(dtype=9), INVALID, "dtype"),
    (dict(x_stride=(-8, 64)), INVALID, "strides"),
    (dict(decay_stride=(64, 4)), UNSUPPORTED, "multiples of 8"),
    (dict(input_stride=(1 << 41, 64)), UNSUPPORTED, "2^40"),
    (dict(seq_len=1 << 20, x_stride=(0, 1 << 40)), UNSUPPORTED, "2^56"),
    (dict(out_stride=(64, 64)), INVALID, "one place"),
    (dict(out_stride=(300 * 64, 56)), INVALID, "one place"),
    (dict(out_stride=(0, 64)), INVALID, "one place"),
]


@pytest.mark.parametrize("kw,status,word", BAD_REC)
def test_gatedrec_refuses_descriptors(kw, status, word):
    d = rec_desc(**kw)
    refused(lambda: seq.ttt_gatedrec_forward(d, at(1), at(2), at(3), at(4), None, None, None, at(5),
                                             None, at(8), 1 << 29, 0), status, word)
    if word != "one place":
        for fn in (seq.ttt_gatedrec_workspace_size, seq.ttt_gatedrec_backward_workspace_size,
                   seq.ttt_gatedrec_saved_size):
            refused(lambda: fn(d), status, word)


def test_gatedrec_refuses_buffers():
    d = rec_desc()
    need = seq.ttt_gatedrec_workspace_size(d)
    assert seq.ttt_gatedrec_saved_size(d) == 2 * 3 * 64 * 4
    # x, decay, input, rate, lengths, state_in, state_out, h, saved
    ok = [at(i) for i in range(1, 10)]
    fwd = lambda a, ws=at(20), n=need: (  # noqa: E731
        lambda: seq.ttt_gatedrec_forward(d, *a, ws, n, 0))
    for i in (0, 1, 2, 3, 7):
        bad = list(ok)
        bad[i] = None
        refused(fwd(bad), INVALID, "non-NULL")
    for i in (0, 1, 2, 3, 5, 6, 7, 8):
        bad = list(ok)
        bad[i] += 8
        refused(fwd(bad), INVALID, "16-byte")
    bad = list(ok)
    bad[4] += 2
    refused(fwd(bad), INVALID, "4-byte")
    for i, j in ((7, 0), (7, 2), (6, 3), (8, 5), (7, 4), (8, 7), (6, 7)):
        bad = list(ok)
        bad[i] = bad[j]
        refused(fwd(bad), INVALID, "overlaps")
    bad = list(ok)
    bad[6] = bad[5] + 64  # in place is the same address or none
    refused(fwd(bad), INVALID, "state_out overlaps state_in")
    if need:
        refused(fwd(ok, None, 0), INVALID, "ws is NULL")
        refused(fwd(ok, at(20) + 16), INVALID, "256-byte")
        refused(fwd(ok, n=need - 1), SMALL, "needed")
        refused(fwd(ok, at(8)), INVALID, "overlaps")


def test_gatedrec_backward_refusals():
    d = rec_desc()
    need = seq.ttt_gatedrec_backward_workspace_size(d)
    # x, decay, input, rate, lengths, saved, dh, dstate_out, dx, ddecay, dinput, drate, dstate_in
    ok = [at(i) for i in range(1, 14)]
    bwd = lambda a, ws=at(20), n=need: (  # noqa: E731
        lambda: seq.ttt_gatedrec_backward(d, *a, ws, n, 0))
    for i in (0, 1, 2, 3, 5, 6, 8, 9, 10, 11):
        bad = list(ok)
        bad[i] = None
        refused(bwd(bad), INVALID, "non-NULL")
    refused(bwd(ok, None, 0), INVALID, "ws is NULL")
    refused(bwd(ok, n=need - 1), SMALL, "needed")
    for i, j in ((8, 0), (9, 1), (10, 2), (8, 9), (11, 3), (12, 5), (10, 6), (11, 4)):
        bad = list(ok)
        bad[i] = bad[j]
        refused(bwd(bad), INVALID, "overlaps")


# ---------------------------------------------------------- activations in 8 bits
def act_desc(**kw):
    return seq.make_act8_desc(**(dict(rows=10, d=64, dtype=torch.bfloat16) | kw))


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=0), INVALID, "rows"),
    (dict(rows=1 << 31), UNSUPPORTED, "rows"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=36), UNSUPPORTED, "d must"),
    (dict(rows=1 << 30, d=2048), UNSUPPORTED, "2^40"),
    (dict(x_stride=56), INVALID, "x_stride"),
    (dict(x_stride=68), UNSUPPORTED, "x_stride"),
    (dict(rows=1 << 30, x_stride=1 << 40), UNSUPPORTED, "2^56"),
    (dict(dtype=5), INVALID, "dtype"),
])
def test_act8_refuses_descriptors(kw, status, word):
    d = act_desc(**kw)
    refused(lambda: seq.ttt_act8_store(d, at(1), at(2), at(3), 0), status, word)
    refused(lambda: seq.ttt_act8_load(d, at(1), at(2), at(3), 0), status, word)


def test_act8_refuses_buffers():
    d = act_desc()
    for fn in (seq.ttt_act8_store, seq.ttt_act8_load):
        for i in range(3):
            bad = [at(1), at(2), at(3)]
            bad[i] = None
            refused(lambda: fn(d, *bad, 0), INVALID, "non-NULL")
        refused(lambda: fn(d, at(1) + 8, at(2), at(3), 0), INVALID, "16-byte")
    store = lambda *a: (lambda: seq.ttt_act8_store(d, *a, 0))  # noqa: E731
    refused(store(at(1), at(1), at(3)), INVALID, "codes overlaps x")
    refused(store(at(1), at(2), at(1) + 3), INVALID, "exps overlaps x")
    refused(store(at(1), at(2) + 8, at(3)), INVALID, "16-byte")
    load = lambda *a: (lambda: seq.ttt_act8_load(d, *a, 0))  # noqa: E731
    refused(load(at(1), at(2), at(1)), INVALID, "x overlaps codes")
    refused(load(at(1), at(2), at(3) + 8), INVALID, "16-byte")
    refused(lambda: seq.ttt_act8_store(d, at(1), at(2), at(2) + 16, 0), INVALID, "exps overlaps codes")
    refused(lambda: seq.ttt_act8_load(d, at(1), at(2), at(2), 0), INVALID, "x overlaps exps")


BAD_WGRAD = [
    (dict(rows=0), INVALID, "rows"),
    (dict(rows=1 << 31), UNSUPPORTED, "rows"),
    (dict(d_in=4), UNSUPPORTED, "d_in"),
    (dict(d_out=0), INVALID, "d_out"),
    (dict(d_out=1 << 21), UNSUPPORTED, "d_out"),
    (dict(rows=1 << 30, d_in=2048), UNSUPPORTED, "rows * d_in"),
    (dict(d_in=1 << 19, d_out=1 << 18), UNSUPPORTED, "2^36"),
    (dict(dy_stride=40), INVALID, "dy_stride"),
    (dict(dy_stride=52), UNSUPPORTED, "dy_stride"),
    (dict(dtype=4), INVALID, "dtype"),
    (dict(dtype=torch.float32, grad_dtype=torch.bfloat16), INVALID, "grad_dtype"),
    (dict(accumulate=3), INVALID, "accumulate"),
    (dict(grad_dtype=torch.bfloat16, accumulate=1), INVALID, "accumulate needs"),
]


def wgrad_desc(**kw):
    return seq.make_act8_wgrad_desc(**(dict(rows=100, d_in=64, d_out=48, dtype=torch.bfloat16) | kw))


@pytest.mark.parametrize("kw,status,word", BAD_WGRAD)
def test_weight_grad_refuses_descriptors(kw, status, word):
    d = wgrad_desc(**kw)
    refused(lambda: seq.ttt_act8_weight_grad_workspace_size(d), status, word)
    refused(lambda: seq.ttt_act8_weight_grad(d, at(1), at(2), at(3), at(4), at(5), 1 << 29, 0),
            status, word)


def test_weight_grad_refuses_buffers():
    d = wgrad_desc()
    need = seq.ttt_act8_weight_grad_workspace_size(d)
    ok = [at(i) for i in range(1, 5)]
    call = lambda a, ws=at(9), n=need: (  # noqa: E731
        lambda: seq.ttt_act8_weight_grad(d, *a, ws, n, 0))
    for i in range(4):
        bad = list(ok)
        bad[i] = None
        refused(call(bad), INVALID, "non-NULL")
    for i in (0, 2, 3):
        bad = list(ok)
        bad[i] += 8
        refused(call(bad), INVALID, "16-byte")
    for j in range(3):
        bad = list(ok)
        bad[3] = bad[j]
        refused(call(bad), INVALID, "grad overlaps")
    if need:
        refused(call(ok, None, 0), INVALID, "ws is NULL")
        refused(call(ok, at(9) + 128), INVALID, "256-byte")
        refused(call(ok, n=need - 1), SMALL, "needed")
        refused(call(ok, at(2)), INVALID, "overlaps")


def test_sizes_need_a_place_to_go():
    lib = seq._load()
    for name, d in (("ttt_embed_backward_workspace_size", embed_desc()),
                    ("ttt_gatedrec_saved_size", rec_desc()),
                    ("ttt_gatedrec_workspace_size", rec_desc()),
                    ("ttt_gatedrec_backward_workspace_size", rec_desc()),
                    ("ttt_act8_weight_grad_workspace_size", wgrad_desc())):
        assert getattr(lib, name)(ctypes.byref(d), None) == INVALID
        n = ctypes.c_size_t(0)
        assert getattr(lib, name)(None, ctypes.byref(n)) == INVALID
        assert getattr(lib, name)(ctypes.byref(d), ctypes.byref(n)) == 0
        assert tm.ttt_last_error() == ""


# ------------------------------------------------------------------ the binding
def test_binding_refuses_tensors():
    ids, t = torch.zeros(3, dtype=torch.int64), torch.zeros(10, 16)
    for bad in (dict(ids=ids.short()), dict(ids=ids.float()), dict(table=t.double()),
                dict(table=t[0]), dict(table=t[:0]), dict(out_dtype=torch.bfloat16),
                dict()):  # CPU tensors
        with pytest.raises(ValueError):
            seq.embed_forward(**(dict(ids=ids, table=t) | bad))
    dout = torch.zeros(3, 16)
    for bad in (dict(dout=dout[:2]), dict(dout=dout.double()), dict(ids=ids.bool()),
                dict(grad=t[:9]), dict(grad=t.bfloat16()), dict(grad_dtype=torch.bfloat16),
                dict(grad=t, grad_dtype=torch.float64), dict()):
        with pytest.raises(ValueError):
            seq.embed_backward(**(dict(dout=dout, ids=ids, vocab=10) | bad))
    x, rate = torch.zeros(2, 5, 16), torch.zeros(16)
    base = dict(x=x, decay_gate=x, input_gate=x, rate=rate)
    bads = (dict(x=x[0]), dict(x=x[:, :0]), dict(x=x.double()), dict(decay_gate=x[:, :4]),
            dict(input_gate=x.bfloat16()), dict(rate=rate[:8]), dict(rate=rate.double()),
            dict(lengths=torch.zeros(2)), dict(lengths=torch.zeros(3, dtype=torch.int32)), dict())
    for bad in bads + (dict(state=torch.zeros(2, 8)), dict(state_out=rate),
                       dict(x=x.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            seq.gatedrec_forward(**(base | bad))
    back = dict(dh=x, saved=torch.zeros(2, 1, 16))
    for bad in bads + (dict(dh=x[:, :3]), dict(dh=x.bfloat16()), dict(saved=None),
                       dict(saved=torch.zeros(2, 2, 16)), dict(dstate_out=torch.zeros(16))):
        with pytest.raises(ValueError):
            seq.gatedrec_backward(**(base | back | bad))
    codes, exps = torch.zeros(4, 40, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    for bad in (torch.zeros(4, 40).double(), torch.zeros(0, 8), torch.tensor(1.0),
                torch.zeros(2, 3, 8).transpose(0, 1), torch.zeros(4, 40)):
        with pytest.raises(ValueError):
            seq.act8_store(bad)
    for bad in (dict(codes=codes.byte()), dict(exps=exps[:3]), dict(exps=exps.char()),
                dict(dtype=torch.float16), dict()):
        with pytest.raises(ValueError):
            seq.act8_load(**(dict(codes=codes, exps=exps) | bad))
    dy = torch.zeros(4, 24)
    for bad in (dict(dy=dy[:3]), dict(dy=dy.double()), dict(dy=dy[:, :0]), dict(exps=exps[:, :1]),
                dict(grad_dtype=torch.bfloat16), dict(grad=torch.zeros(24, 40)),
                dict(grad=torch.zeros(40, 24).bfloat16()), dict()):
        with pytest.raises(ValueError):
            seq.act8_weight_grad(**(dict(codes=codes, exps=exps, dy=dy) | bad))


def test_calls_without_tokens():
    e = torch.zeros(0, dtype=torch.int64)
    assert seq.embed_forward(e, torch.zeros(10, 16)).shape == (0, 16)
    g = seq.embed_backward(torch.zeros(0, 16), e, 10)
    assert g.shape == (10, 16) and not g.any()
    keep = torch.ones(10, 16)
    assert seq.embed_backward(torch.zeros(0, 16), e, 10, grad=keep) is keep and keep.all()


def test_a_scale_counts_with_its_value(monkeypatch):
    seen = []
    monkeypatch.setattr(seq, "ttt_embed_forward", lambda d, *a, **k: seen.append(d.scale))
    monkeypatch.setattr(seq, "ttt_embed_backward", lambda d, *a, **k: seen.append(d.scale))
    ids, t = torch.zeros(3, dtype=torch.int64), torch.zeros(10, 16)
    s = torch.tensor(0.5)
    for v in (0.5, 2.0):
        s.fill_(v)
        seq.embed_forward(ids, t, s)
        assert seen.pop() == v
        seq.embed_backward(torch.zeros(3, 16), ids, 10, s)
        assert seen.pop() == v


def test_streams_and_workspaces_given(monkeypatch):
    """A stream given as a handle is the one that a call runs and allocates on; a workspace is
    looked at like every other tensor."""
    entered, looked = [], []
    monkeypatch.setattr(seq, "_on", lambda s, like: entered.append(s) or contextlib.nullcontext())
    monkeypatch.setattr(seq, "_same_device", lambda like, *t: looked.extend(t))
    for name in ("ttt_embed_forward", "ttt_embed_backward", "ttt_gatedrec_forward",
                 "ttt_gatedrec_backward", "ttt_act8_store", "ttt_act8_load",
                 "ttt_act8_weight_grad"):
        monkeypatch.setattr(seq, name, lambda *a, **k: None)
    ids, t, ws = torch.zeros(3, dtype=torch.int64), torch.zeros(10, 16), torch.zeros(256)
    x, rate = torch.zeros(2, 5, 16), torch.zeros(16)
    codes, exps = torch.zeros(4, 40, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    calls = (lambda **k: seq.embed_backward(torch.zeros(3, 16), ids, 10, **k),
             lambda **k: seq.gatedrec_forward(x, x, x, rate, **k),
             lambda **k: seq.gatedrec_backward(x, x, x, rate, x, torch.zeros(2, 1, 16), **k),
             lambda **k: seq.act8_weight_grad(codes, exps, torch.zeros(4, 24), **k))
    for call in calls:
        call(ws=ws)
        assert any(q is ws for q in looked)
        looked.clear()
    for call in calls + (lambda **k: seq.embed_forward(ids, t, **k), lambda **k: seq.act8_store(t, **k),
                         lambda **k: seq.act8_load(codes, exps, **k)):
        call(stream=0)
        assert entered.pop() == 0 and not entered


# ------------------------------------------------ the 64-bit forms against differences
def test_gatedrec_reference_against_differences():
    rng = np.random.default_rng(3)
    B, T, d = 2, 6, 5
    n = rng.normal
    x, dg, ig, dh = (n(size=(B, T, d)) for _ in range(4))
    rate, st, ds, ln = rng.uniform(0.1, 2, size=d), n(size=(B, d)), n(size=(B, d)), [6, 4]
    dh[1, 4:] = 0
    grads = ref.gatedrec_grads(x, dg, ig, rate, dh, st, ds, ln)

    def f(*a):
        h, S = ref.gatedrec(*a[:4], a[4], ln)
        return (dh * h).sum() + (ds * S).sum()

    e = 1e-6
    args = [x, dg, ig, rate, st]
    for i, g in enumerate(grads):
        u = n(size=args[i].shape)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + e * u, args[i] - e * u
        # third derivatives times e^2 and 2^-52 / e: both far below
        assert abs((f(*hi) - f(*lo)) / (2 * e) - (g * u).sum()) < 1e-8 * max(1, np.abs(g * u).sum())


def test_act8_reference():
    x = np.array([[127.0] + [0] * 31 + [127.01] + [0.5] * 7, [0.0] * 40])
    codes, exps = ref.act8(x)
    assert exps.tolist() == [[127, 128], [1, 1]]
    assert codes[0, 0] == 127 and codes[0, 32] == 64 and (codes[0, 33:] == 0).all()
    v = ref.act8_value(codes, exps)
    assert v[0, 0] == 127 and v[0, 32] == 128 and not v[1].any()
    x[1, 3] = np.nan
    codes, exps = ref.act8(x)
    assert exps[1, 0] == 255 and np.isnan(ref.act8_value(codes, exps)[1, :32]).all()


# ---------------------------------------------------- the waits of the compiled kernels


def kernels_of(source, tmp_path):
    """{name: lines} of the gfx950 code that build.py's own compiler and flags make."""
    out = tmp_path / (source + ".s")
    flags = [f for f in hipbuild.HIPCC_FLAGS if f != "-shared"]
    cmd = [hipbuild.hipcc(), *flags, "--cuda-device-only", "-S",
           os.path.join(hipbuild.CSRC, source), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    parts = re.split(r"^(?=_Z\w+:)", out.read_text(), flags=re.M)[1:]
    return {p.split(":", 1)[0]: p.split(".Lfunc_end")[0].splitlines() for p in parts}


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_no_load_into_lds_is_in_flight_at_a_barrier(tmp_path):
    """The products fill LDS tiles by direct loads and let other waves read them after a barrier:
    vmcnt(0) stands between a direct load and the next barrier, in the order of the code (whose
    loops end with no load in flight); and every transposing read has its own wait behind it, in
    the same block."""
    found = barriers = reads = 0
    for name, lines in kernels_of("act8.hip", tmp_path).items():
        if not any(re.search(r"buffer_load\w* .*\blds$", x) for x in lines):
            continue
        found += 1
        assert not any("scratch_" in x for x in lines), name  # nothing spilled either
        flying, pending = False, 0
        for x in lines:
            if "ds_read_b64_tr_b16" in x:
                pending += 1
                reads += 1
            elif pending and re.search(r"s_waitcnt.*lgkmcnt\(0\)", x):
                pending = 0
            elif pending:
                assert "mfma" not in x and "s_barrier" not in x, (name, x)
            if re.search(r"buffer_load\w* .*\blds$", x):
                flying = True
            elif re.search(r"s_waitcnt.*vmcnt\(0\)", x):
                flying = False
            elif "s_barrier" in x:
                assert not flying, (name, x)
                barriers += "s_barrier" in x
        assert not flying, name
    assert found == 9 and barriers >= 3 * found and reads >= 4 * 4, (found, barriers, reads)


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")
def test_no_packed_arithmetic(tmp_path):
    for source in ("embed.hip", "gatedrec.hip", "act8.hip"):
        for name, lines in kernels_of(source, tmp_path).items():
            assert not any(re.search(r"v_pk_(add|mul|fma)_f32", x) for x in lines), name


# ------------------------------------------- the recurrence's links, on the CPU
def test_the_state_found_does_not_depend_on_when_it_is_looked_for():
    """state_before of gatedrec.hip, its steps in Python: whatever part of the groups of tiles in
    front has published its state, its map or nothing, what is found is the same number to the
    bit, or nothing yet; and with every group in front published something is found."""
    rng = np.random.default_rng(7)
    f32 = np.float32
    kAhead = 6

    def apply(dec, h, u):
        near = np.signbit(dec)
        return f32(f32(f32(np.float64(dec) * np.float64(h) + np.float64(u)))
                   + (h if near else f32(0)))

    n = 30
    dec = [f32(-abs(rng.normal()) * 0.1) if rng.random() < 0.5 else f32(rng.random() * 0.7)
           for _ in range(n)]
    u = [f32(rng.normal()) for _ in range(n)]
    states, s = [], f32(rng.normal())
    for j in range(n):  # behind group j
        s = apply(dec[j], s, u[j])
        states.append(s)

    def look(k, word):
        found, s = False, f32(0)
        for i in reversed(range(kAhead)):
            kind, d, h = word[k - 1 - min(i, k - 1)]
            found = kind == "state" or (found and kind != "unset")
            s = h if kind == "state" else apply(d, s, h) if kind == "map" else s
        return s if found else None

    for k in range(1, n):
        for _ in range(50):
            word = []
            for j in range(n):
                kind = rng.choice(["unset", "map", "state"])
                if j == 0 and kind == "map":
                    kind = "state"  # the first group's word has no map
                word.append((kind, dec[j], states[j] if kind == "state" else u[j]))
            got = look(k, word)
            assert got is None or got == states[k - 1]
    # maps alone behind the first group's state: found as far as kAhead reaches, then in turn
    word = [("state", None, states[0])] + [("map", dec[j], u[j]) for j in range(1, n)]
    for j in range(1, n):
        before = look(j, word)
        assert before is not None and before == states[j - 1]
        word[j] = ("state", None, apply(dec[j], before, u[j]))


def test_the_decay_over_two_runs():
    """decay_both of gatedrec.hip, its steps in Python: a decay near 1 is kept as its distance from
    1 (sign bit set), the product of any two to 2^-22 of itself and, near 1, of its distance."""
    f32 = np.float32

    def fma(a, b, c):
        return f32(np.float64(a) * np.float64(b) + np.float64(c))

    def both(d1, d2):
        n1, n2 = np.signbit(d1), np.signbit(d2)
        near = -abs(fma(d1, d2, f32(d1 + d2)))
        if n1 and n2:
            return f32(f32(1) + near) if near < -0.5 else near
        return fma(d1, d2, d2 if n1 else d1 if n2 else f32(0))

    def value(d):  # (a, 1 - a)
        return (1 + np.float64(d), -np.float64(d)) if np.signbit(d) else (np.float64(d), 1 - np.float64(d))

    rng = np.random.default_rng(8)
    one = f32(-0.0)
    some = [one, f32(0), f32(1e-30), f32(0.7), f32(-0.29), f32(-1e-7), f32(-1e-30)]
    some += [f32(-(10.0 ** -e)) for e in rng.uniform(0.6, 8, 40)] + [f32(x) for x in rng.uniform(0, .7, 40)]
    for a in some:
        assert value(both(one, a)) == value(a) and np.signbit(both(one, a)) == np.signbit(a)
        assert value(both(a, one)) == value(a)
        for b in some:
            got = both(a, b)
            (va, ua), (vb, ub) = value(a), value(b)
            # (below fp32's smallest, 2^-149, a product rounds to it or to 0)
            assert abs(value(got)[0] - va * vb) <= 2.0 ** -22 * va * vb + 2.0 ** -149
            if np.signbit(got):  # 1 - a b = (1 - a) + (1 - b) - (1 - a)(1 - b)
                want = ua + ub - ua * ub
                assert abs(value(got)[1] - want) <= 2.0 ** -22 * want + 2.0 ** -149
    nan = f32("nan")
    assert np.isnan(both(nan, one)) and np.isnan(both(one, nan)) and np.isnan(both(f32(0.5), nan))
