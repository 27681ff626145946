"""The block operators on the GPU against their 64-bit forms: residual addition
with the RMS norm, linear attention with a decay for each head, and their
gradients, at the sizes, strides, masks and values where they can go wrong.

Tolerances (relative Frobenius), from the number formats:
  fp32: each result is a sum of products with relative rounding 2^-24 a term, at
        most some hundred of them one after the other: 2e-6 (2^-24 times 32);
  bf16 result of fp32 arithmetic: one rounding, at most 2^-8 a value: 2^-8;
  bf16 result of the chunked form: the scores, the state's copy and the result
        are each rounded once, at most 2^-8 a value each: the scores' and the
        copy's parts add to one result, 2 * 2^-8;
  fp32 state of the chunked form from bf16: the weighted values go in as a sum
        of bf16 terms, at most 2^-17 a value: 2^-16 (1.5e-5);
  8-bit result: 2^-4 a value (half of the last of 3 mantissa bits), times its
        scale; below 2^-6 of the scaled range the spacing is 2^-9, half of it 2^-10.
"""
import numpy as np
import pytest
import torch

from chunk_wise_weight_chunked_amd import block
from chunk_wise_weight_chunked_amd import ttt_mlp as tm

import _block_ref as ref
from _block_ref import f64, rel

pytestmark = pytest.mark.gpu

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TOL_F32 = 2e-6
TOL_ROUND = {F32: TOL_F32, BF16: 2.0 ** -8}
TOL_CHUNK = {F32: TOL_F32, BF16: 2.0 ** -7}
TOL_STATE = {F32: TOL_F32, BF16: 2.0 ** -16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tm.load()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def say(*a):
    print(*a, flush=True)


# ------------------------------------------------------------------- the norm
NORM_SHAPES = [(1, 8), (3, 64), (33, 128), (17, 136), (5, 512), (700, 520), (9, 1024), (513, 2560),
               (7, 2560), (600, 4096), (5, 4104), (3, 9728), (2, 16384)]


@pytest.mark.parametrize("dtype,res_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,d", NORM_SHAPES)
def test_norm_forward(rows, d, dtype, res_dtype):
    say(rows, d, dtype, res_dtype)
    g = gen(rows * 7 + d)
    x, w = normal(g, rows, d, dtype=dtype), normal(g, d, dtype=dtype)
    res = normal(g, rows, d, dtype=res_dtype, std=3.0)
    r64, y64 = ref.addnorm(f64(x), f64(res), f64(w), 1e-6)
    y, r, scale = block.add_rmsnorm(x, res, w)
    assert scale is None and r.dtype == res_dtype and y.dtype == dtype
    assert rel(f64(r), r64) <= TOL_ROUND[res_dtype]
    assert rel(f64(y), y64) <= TOL_ROUND[dtype]
    y0, r0, _ = block.add_rmsnorm(x, None, w)
    assert r0 is None
    assert rel(f64(y0), ref.addnorm(f64(x), None, f64(w), 1e-6)[1]) <= TOL_ROUND[dtype]
    # the residual updated in place
    y1, r1, _ = block.add_rmsnorm(x, res, w, r_out=res)
    assert r1 is res and torch.equal(r1, r) and torch.equal(y1, y)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", [(1, 128), (9, 256), (600, 640), (5, 2560), (513, 2560), (3, 8192)])
def test_norm_fp8(rows, d, dtype, group):
    say(rows, d, dtype, group)
    g = gen(rows + d)
    x, res = normal(g, rows, d, dtype=dtype), normal(g, rows, d)
    w = normal(g, d, dtype=dtype)
    x[0] = 0
    res[0] = 0  # a row of zeros: scale 1, values 0
    y, r, scale = block.add_rmsnorm(x, res, w, out_dtype=FP8, scale_group=group)
    _, y64 = ref.addnorm(f64(x), f64(res), f64(w), 1e-6)
    n = d // (group or d)
    assert y.dtype == FP8 and scale.shape == (rows, n)
    top = np.abs(y64).reshape(rows, n, -1).max(-1)
    want = np.where(top > 0, top / 448.0, 1.0)
    assert np.allclose(f64(scale), want, rtol=2e-6, atol=0)
    got = f64(y.float()).reshape(rows, n, -1) * f64(scale)[..., None]
    near = np.abs(got - y64.reshape(rows, n, -1))
    bound = np.maximum(2.0 ** -4 * np.abs(y64.reshape(rows, n, -1)), 2.0 ** -10 * want[..., None])
    assert (near <= bound * (1 + 1e-4)).all()
    assert torch.equal(y[0].float(), torch.zeros(d, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_fp8_smallest_values(group, dtype):
    """Values whose scale would have no finite reciprocal: a run beside ordinary ones, a row."""
    d = 256
    x = torch.ones(3, d, device="cuda")
    x[0, 128:] = torch.linspace(-1e-38, 1e-38, 128)
    x[1, 128:] = 2.0 ** -133  # the smallest bf16
    w = torch.ones(d, device="cuda")
    for w in (w, w * 1e-38):
        a, b = x.to(dtype), w.to(dtype)
        y, _, scale = block.add_rmsnorm(a, None, b, out_dtype=FP8, scale_group=group)
        _, y64 = ref.addnorm(f64(a), None, f64(b), 1e-6)
        s = f64(scale)
        y64, got = y64.reshape(3, s.shape[1], -1), f64(y.float()).reshape(3, s.shape[1], -1)
        assert np.isfinite(got).all() and (s >= 2.0 ** -126).all()
        # and fp32's own smallest step, on the values before the scale
        bound = np.maximum(2.0 ** -4 * np.abs(y64), 2.0 ** -10 * s[..., None]) * (1 + 1e-4) + 2.0 ** -149
        assert (np.abs(got * s[..., None] - y64) <= bound).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,d", [(600, 128), (257, 512), (2100, 1024), (513, 2560), (40, 16384)])
def test_norm_fp8_codes(rows, d, group):
    """The stored codes are y / scale rounded to nearest even, y the fp32 norm: the same that the
    call without 8 bits gives for fp32 rows, divided and rounded here."""
    g = gen(rows)
    x, res, w = normal(g, rows, d), normal(g, rows, d), normal(g, d)
    y, _, _ = block.add_rmsnorm(x, res, w)
    q, _, scale = block.add_rmsnorm(x, res, w, out_dtype=FP8, scale_group=group)
    n = d // (group or d)
    y = f64(y).astype(np.float32).reshape(rows, n, -1)
    top = np.abs(y).max(-1, keepdims=True)
    s = f64(scale).astype(np.float32).reshape(rows, n, 1)
    assert np.array_equal(s, top / np.float32(448))
    codes = torch.from_numpy(y / s).to(FP8).float().numpy()  # numpy's division is rounded once
    wrong = int((f64(q.float()).reshape(codes.shape) != codes).sum())
    assert wrong == 0, f"{wrong} of {codes.size}"


def test_norm_strides_and_in_place():
    g = gen(3)
    wide = normal(g, 40, 3 * 256, dtype=BF16)
    x, w = wide[:, 256:512], normal(g, 256, dtype=BF16)
    y, _, _ = block.add_rmsnorm(x, None, w)
    y0, _, _ = block.add_rmsnorm(x.contiguous(), None, w)
    assert torch.equal(y, y0)
    keep = wide.clone()
    desc = block.make_addnorm_desc(40, 256, BF16, x_stride=768, y_stride=768)
    block.ttt_addnorm_forward(desc, x, None, w, None, x)  # y over x, in the wide rows
    assert torch.equal(wide[:, 256:512], y0)
    assert torch.equal(wide[:, :256], keep[:, :256]) and torch.equal(wide[:, 512:], keep[:, 512:])


def test_norm_rows_beyond_one_launch():
    """More rows than one launch's threads: the rows at the seams and the ends, every output."""
    rows, d = (1 << 28) + 5, 8
    x = torch.empty(rows, d, dtype=BF16, device="cuda").normal_()
    res = torch.empty(rows, d, dtype=BF16, device="cuda").normal_()
    w = normal(gen(4), d, dtype=BF16)
    look = torch.cat([torch.arange(s - 40, s + 40) for s in (40, 1 << 27, 1 << 28)]
                     + [torch.arange(rows - 9, rows)]).clamp(max=rows - 1).unique().cuda()
    r64, y64 = ref.addnorm(f64(x[look]), f64(res[look]), f64(w), 1e-6)
    y, r, scale = block.add_rmsnorm(x, res, w, out_dtype=FP8)
    assert rel(f64(r[look]), r64) <= TOL_ROUND[BF16]
    top = np.abs(y64).max(-1)
    assert np.allclose(f64(scale[look]).reshape(-1), np.where(top > 0, top / 448.0, 1.0), rtol=2e-6, atol=0)
    near = np.abs(f64(y[look].float()) * f64(scale[look]).reshape(-1, 1) - y64)
    assert (near <= np.maximum(2.0 ** -4 * np.abs(y64), 2.0 ** -10 * top[:, None] / 448) * (1 + 1e-4)).all()
    del y, scale, r, res
    _, y64 = ref.addnorm(f64(x[look]), None, f64(w), 1e-6)
    desc = block.make_addnorm_desc(rows, d, BF16)
    block.ttt_addnorm_forward(desc, x, None, w, None, x)
    assert rel(f64(x[look]), y64) <= TOL_ROUND[BF16]


def test_norm_values_out_of_the_ordinary():
    x = torch.zeros(5, 256, device="cuda")
    x[1] = 3e19          # the sum of squares overflows: 1 / sqrt(inf) = 0
    x[2, 3] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 1e-20         # eps holds the root up
    w = torch.ones(256, device="cuda")
    y, _, _ = block.add_rmsnorm(x, None, w)
    assert (y[0] == 0).all() and (y[1] == 0).all() and torch.isnan(y[3]).all()
    assert torch.isnan(y[2, 3]) and (y[2, :3] == 0).all()
    assert rel(f64(y[4]), np.full(256, 1e-17)) <= 1e-6
    z, _, _ = block.add_rmsnorm(torch.zeros(1, 64, device="cuda"), None,
                                torch.ones(64, device="cuda"), eps=0.0)
    assert torch.isnan(z).all()  # 0 / 0 without an eps, as the formula says


@pytest.mark.parametrize("dtype,res_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,d", [(1, 8), (37, 128), (65, 136), (2100, 256), (300, 2560),
                                    (2600, 1024), (9, 4104), (3, 16384)])
def test_norm_backward(rows, d, dtype, res_dtype):
    say(rows, d, dtype, res_dtype)
    g = gen(rows * 3 + d)
    r, dy = normal(g, rows, d, dtype=res_dtype, std=2.0), normal(g, rows, d, dtype=dtype)
    w, dro = normal(g, d, dtype=dtype), normal(g, rows, d, dtype=res_dtype)
    for extra in (None, dro):
        dr, dx, dw = block.add_rmsnorm_backward(dy, r, w, dr=extra)
        want, want_w = ref.addnorm_grads(f64(dy), f64(r), f64(w), 1e-6, f64(extra))
        assert rel(f64(dr), want) <= TOL_ROUND[res_dtype]
        assert rel(f64(dx), want) <= TOL_ROUND[dtype] and dx.dtype == dtype
        assert rel(f64(dw), want_w) <= TOL_F32
    again = block.add_rmsnorm_backward(dy, r, w, dr=dro)
    assert all(torch.equal(a, b) for a, b in zip(again, (dr, dx, dw)))
    desc = block.make_addnorm_desc(rows, d, dtype, res_dtype)
    block.ttt_addnorm_backward(desc, dy, r, w, dro, dro, None, None)  # no dw, dr in place
    assert torch.equal(dro, dr)


def test_norm_backward_against_differences():
    g = gen(11)
    r, dy, w = normal(g, 12, 512), normal(g, 12, 512), normal(g, 512)
    u, z = normal(g, 12, 512), normal(g, 512)
    dr, _, dw = block.add_rmsnorm_backward(dy, r, w)
    e = 2.0 ** -7
    f = lambda s: (dy.double() * block.add_rmsnorm(r + s * u, None, w + s * z)[0].double()).sum()  # noqa: E731
    diff = float((f(e) - f(-e)) / (2 * e))
    want = float((dr.double() * u).sum() + (dw.double() * z).sum())
    # third derivatives: e^2 = 6e-5; rounding 2^-24 / e = 8e-6, of sums of size |dy| |y|
    assert abs(diff - want) <= 1e-4 * float(dy.double().norm() * u.double().norm())


# ---------------------------------------------------------- linear attention
# (B, T, H, G, dk, dv): up to 4 tokens in the recurrent form; whole and partial
# chunks of 32; one or more segments; every tile width
ATTN_SHAPES = [(1, 1, 1, 1, 8, 8), (3, 1, 4, 4, 128, 128), (2, 4, 4, 2, 72, 40), (3, 3, 2, 1, 40, 128), (2, 8, 4, 2, 72, 40), (1, 5, 2, 1, 64, 128),
               (1, 9, 1, 1, 16, 8), (2, 31, 2, 1, 64, 64), (1, 32, 3, 3, 128, 64),
               (2, 33, 4, 1, 64, 128), (1, 65, 2, 2, 128, 128), (1, 100, 2, 1, 80, 72),
               (1, 257, 2, 2, 96, 104), (2, 511, 1, 1, 128, 128), (1, 523, 4, 2, 64, 64),
               (1, 1100, 2, 1, 64, 72)]


def attn_inputs(B, T, H, G, dk, dv, dtype, seed):
    g = gen(seed)
    q, k, v = (normal(g, B, T, n, d, dtype=dtype) for n, d in ((H, dk), (G, dk), (G, dv)))
    lg = -torch.exp2(-1.0 - 8.0 * torch.rand(H, generator=g)).cuda()
    st = normal(g, B, H, dk, dv)
    return g, q, k, v, lg, st


def tol_o(dtype, T):
    return TOL_ROUND[dtype] if T <= 8 else TOL_CHUNK[dtype]


def tol_s(dtype, T):
    return TOL_F32 if T <= 8 else TOL_STATE[dtype]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", ATTN_SHAPES, ids=str)
def test_attention_forward(shape, dtype):
    say(shape, dtype)
    B, T, H, G, dk, dv = shape
    _, q, k, v, lg, st = attn_inputs(*shape, dtype, T + dk)
    for state in (None, st):
        o, S = block.linattn_forward(q, k, v, lg, scale=0.3, state=state)
        o64, S64 = ref.linattn(f64(q), f64(k), f64(v), f64(lg), 0.3, f64(state))
        eo, es = rel(f64(o), o64), rel(f64(S), S64)
        say("  o %.2e state %.2e" % (eo, es))
        assert o.dtype == dtype and eo <= tol_o(dtype, T) and es <= tol_s(dtype, T)
    # in place, and without a state out
    keep = st.clone()
    o2, S2 = block.linattn_forward(q, k, v, lg, scale=0.3, state=keep, state_out=keep)
    assert S2 is keep and torch.equal(keep, S) and torch.equal(o2, o)
    desc = block.make_linattn_desc(B, T, H, G, dk, dv, dtype, 0.3)
    ws = torch.empty(block.ttt_linattn_workspace_size(desc) or 1, dtype=torch.uint8, device="cuda")
    o3 = torch.full_like(o, 7.0)
    block.ttt_linattn_forward(desc, q, k, v, lg, None, st, None, o3, ws)
    assert torch.equal(o3, o)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 40, 600])
def test_attention_lengths(T, dtype):
    lens = [0, 1, T - 1, T, T + 5, -3, T // 2, 33]
    B, H, G, dk, dv = len(lens), 2, 1, 64, 40
    _, q, k, v, lg, st = attn_inputs(B, T, H, G, dk, dv, dtype, T)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = ln.clamp(0, T)
    # what lies behind a sequence's end must not be read into anything
    behind = torch.arange(T, device="cuda")[None, :] >= n[:, None]
    for i, t in enumerate((q, k, v)):
        t[behind] = (float("nan"), float("inf"), torch.finfo(dtype).min)[i]
    clean = [torch.where(behind[..., None, None], torch.zeros_like(t), t) for t in (q, k, v)]
    for state in (None, st):
        o, S = block.linattn_forward(q, k, v, lg, state=state, lengths=ln)
        o64, S64 = ref.linattn(*(f64(t) for t in clean), f64(lg), dk ** -0.5, f64(state), lens)
        assert (o[behind] == 0).all()
        assert rel(f64(o), o64) <= tol_o(dtype, T) and rel(f64(S), S64) <= tol_s(dtype, T)
        if state is not None:
            assert torch.equal(S[0], st[0]) and torch.equal(S[5], st[5])  # no tokens
    g = gen(5)
    dO, ds = normal(g, B, T, H, dv, dtype=dtype), normal(g, B, H, dk, dv)
    dO[behind] = float("nan")
    got = block.linattn_backward(q, k, v, lg, dO, state=st, dstate_out=ds, lengths=ln)
    dOc = torch.where(behind[..., None, None], torch.zeros_like(dO), dO)
    want = ref.linattn_grads(*(f64(t) for t in clean), f64(lg), dk ** -0.5, f64(dOc), f64(st),
                             f64(ds), lens)
    for name, w in zip("qkv", want):
        assert (got[name][behind] == 0).all()
        assert rel(f64(got[name]), w) <= TOL_CHUNK[dtype], name
    assert rel(f64(got["state"]), want[3]) <= TOL_STATE[dtype]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (2, 7, 4, 2, 64, 40), (2, 32, 2, 2, 64, 64),
                                   (1, 45, 4, 1, 128, 64), (1, 129, 2, 1, 72, 128),
                                   (2, 300, 2, 2, 128, 128), (1, 777, 3, 1, 64, 96)], ids=str)
def test_attention_backward(shape, dtype):
    say(shape, dtype)
    B, T, H, G, dk, dv = shape
    g, q, k, v, lg, st = attn_inputs(*shape, dtype, T + dv)
    dO, ds = normal(g, B, T, H, dv, dtype=dtype), normal(g, B, H, dk, dv)
    for state, dstate in ((None, None), (st, ds)):
        got = block.linattn_backward(q, k, v, lg, dO, scale=0.3, state=state, dstate_out=dstate)
        want = ref.linattn_grads(f64(q), f64(k), f64(v), f64(lg), 0.3, f64(dO), f64(state),
                                 f64(dstate))
        err = [rel(f64(got[n]), w) for n, w in zip("qkv", want)]
        say("  dq %.2e dk %.2e dv %.2e" % tuple(err))
        assert all(e <= TOL_CHUNK[dtype] for e in err)
        assert (got["state"] is None) == (state is None)
    assert rel(f64(got["state"]), want[3]) <= TOL_STATE[dtype]
    # the state's gradient in place of the one that came in, and results that repeat
    again = block.linattn_backward(q, k, v, lg, dO, scale=0.3, state=st, dstate_out=ds)
    assert all(torch.equal(again[n], got[n]) for n in got)
    desc = block.make_linattn_desc(B, T, H, G, dk, dv, dtype, 0.3)
    ws = torch.empty(block.ttt_linattn_backward_workspace_size(desc) or 1, dtype=torch.uint8,
                     device="cuda")
    block.ttt_linattn_backward(desc, q, k, v, lg, None, st, dO, ds, again["q"], again["k"],
                               again["v"], ds, ws)
    assert torch.equal(ds, got["state"])


def test_attention_backward_against_differences():
    # the operator is linear in each of its inputs: differences are exact but for
    # fp32 rounding, 2^-24 a term of sums of about |dO| |o| (TOL_F32 covers 32 of them)
    B, T, H, G, dk, dv = 2, 90, 4, 2, 64, 40
    g, q, k, v, lg, st = attn_inputs(B, T, H, G, dk, dv, F32, 1)
    dO, ds = normal(g, B, T, H, dv), normal(g, B, H, dk, dv)
    got = block.linattn_backward(q, k, v, lg, dO, state=st, dstate_out=ds)

    def f(a):
        o, S = block.linattn_forward(*a[:3], lg, state=a[3])
        return (dO.double() * o).sum() + (ds.double() * S).sum(), o, S

    for i, name in enumerate(("q", "k", "v", "state")):
        a = [q, k, v, st]
        u = normal(g, *a[i].shape)
        hi, lo = list(a), list(a)
        hi[i], lo[i] = a[i] + u, a[i] - u
        (fh, o, S), (fl, _, _) = f(hi), f(lo)
        size = float(dO.double().norm() * o.double().norm() + ds.double().norm() * S.double().norm())
        assert abs(float(fh - fl) / 2 - float((got[name].double() * u).sum())) <= TOL_F32 * size, name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H", [(2, 1030, 128), (2, 1024, 129), (7, 1100, 40), (16, 1030, 20),
                                   (16, 1024, 32), (64, 1024, 16), (65, 1024, 4), (3, 2100, 60)])
def test_attention_lengths_many_sequences(B, T, H, dtype):
    """Batches whose workgroups are placed by the sequences' lengths: every sequence and head as
    in a call of the sequence alone that has no lengths."""
    say(B, T, H, dtype)
    G, dk, dv = H // (2 if H % 2 == 0 else 1), 8, 16
    g, q, k, v, lg, st = attn_inputs(B, T, H, G, dk, dv, dtype, B + T)
    ln = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    ln[0], ln[-1], ln[B // 2] = T, 0, int(ln[1])  # equal ones too
    dO = normal(g, B, T, H, dv, dtype=dtype)
    o, S = block.linattn_forward(q, k, v, lg, state=st, lengths=ln.cuda())
    d = block.linattn_backward(q, k, v, lg, dO, state=st, lengths=ln.cuda())
    for b in range(B):
        n = int(ln[b])
        assert (o[b, n:] == 0).all() and all((d[x][b, n:] == 0).all() for x in "qkv")
        if n == 0:
            assert torch.equal(S[b], st[b])
            continue
        one = [t[b:b + 1, :n].contiguous() for t in (q, k, v, dO)]
        o1, S1 = block.linattn_forward(*one[:3], lg, state=st[b:b + 1])
        d1 = block.linattn_backward(*one[:3], lg, one[3], state=st[b:b + 1])
        pairs = [(o[b, :n], o1[0], TOL_CHUNK), (S[b], S1[0], TOL_STATE), (d["state"][b], d1["state"][0], TOL_STATE)]
        pairs += [(d[x][b, :n], d1[x][0], TOL_CHUNK) for x in "qkv"]
        for i, (got, want, tol) in enumerate(pairs):  # two results, each within its tolerance
            assert rel(f64(got), f64(want)) <= 2 * tol[dtype], (b, n, i)


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("dv", [8, 128])
def test_attention_most_heads(T, dv):
    """The most heads a call may have, every sequence the same one: as a call of one sequence."""
    B, H, dk = 1 << 17, 16, 8
    _, q, k, v, lg, _ = attn_inputs(1, T, H, H, dk, dv, BF16, 3)
    dO = normal(gen(6), 1, T, H, dv, dtype=BF16)
    want, _ = block.linattn_forward(q, k, v, lg)
    many = [t.expand(B, *t.shape[1:]) for t in (q, k, v)]
    o, _ = block.linattn_forward(*many, lg)
    assert (o == want).all()
    if dv == 8:
        d = block.linattn_backward(*many, lg, dO.expand(B, T, H, dv))
        d1 = block.linattn_backward(q, k, v, lg, dO)
        assert all((d[n] == d1[n]).all() for n in "qkv")


def test_attention_decays():
    # no decay, a memory of thousands of tokens, of one, none at all
    T, dk, dv = 700, 64, 64
    lg = torch.tensor([0.0, -1e-4, -0.02, -3.0, -90.0, -float("inf")], device="cuda")
    H = len(lg)
    for dtype in (BF16, F32):
        for n in (T, 6):
            g, q, k, v, _, st = attn_inputs(1, n, H, H, dk, dv, dtype, 9)
            o, S = block.linattn_forward(q, k, v, lg, state=st)
            with np.errstate(all="ignore"):
                o64, S64 = ref.linattn(f64(q), f64(k), f64(v), f64(lg), dk ** -0.5, f64(st))
            for h in range(H):
                assert rel(f64(o[:, :, h]), o64[:, :, h]) <= tol_o(dtype, n), (dtype, n, h)
                assert rel(f64(S[:, h]), S64[:, h]) <= tol_s(dtype, n), (dtype, n, h)
        dO = normal(g, 1, T, H, dv, dtype=dtype)
        _, q, k, v, _, st = attn_inputs(1, T, H, H, dk, dv, dtype, 10)
        got = block.linattn_backward(q, k, v, lg, dO, state=st)
        want = ref.linattn_grads(f64(q), f64(k), f64(v), f64(lg), dk ** -0.5, f64(dO), f64(st))
        for name, w in zip("qkv", want):
            for h in range(H):
                assert rel(f64(got[name][:, :, h]), w[:, :, h]) <= TOL_CHUNK[dtype], (name, h)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dv", [64, 96])
def test_attention_large_states_decay_to_nothing(dv, dtype):
    """A state of 1e36 that comes in, and nothing else: with decays of exp(-1) and below it is 0 in
    fp32 (below 2^-149) for every token from 190 on, whatever segments the tokens are in."""
    B, T, H, G, dk = 1, 4096, 64, 1, 64
    g, q, k, v, _, _ = attn_inputs(B, T, H, G, dk, dv, dtype, 15)
    lg = torch.linspace(-1.0, -20.0, H, device="cuda")
    st = torch.full((B, H, dk, dv), 1e36, device="cuda")
    none = lambda t: torch.zeros_like(t)  # noqa: E731
    o, S = block.linattn_forward(q, none(k), v, lg, state=st)
    assert (o[:, 190:] == 0).all() and (S == 0).all() and (o[:, 0] != 0).any()
    dO = torch.zeros(B, T, H, dv, dtype=dtype, device="cuda")
    d = block.linattn_backward(q, k, v, lg, dO, state=st, dstate_out=st)
    assert (d["k"][:, :T - 190] == 0).all() and (d["v"][:, :T - 190] == 0).all()
    assert (d["k"][:, T - 1] != 0).any() and (d["state"] == 0).all()
    dO = normal(g, B, T, H, dv, dtype=dtype)
    assert (block.linattn_backward(q, none(k), v, lg, dO, state=st)["q"][:, 190:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 29, 70, 600])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_attention_infinities_stay_behind_the_mask(T, bad, dtype):
    """An infinity or NaN at token s reaches only the results that the formula gives it to: the
    others are those of a call without it, bit for bit."""
    H, G, dk, dv = 2, 1, 64, 72
    g, q, k, v, _, st = attn_inputs(1, T, H, G, dk, dv, dtype, T)
    lg = torch.tensor([-1e-3, -0.5], device="cuda")
    dO, ds = normal(g, 1, T, H, dv, dtype=dtype), normal(g, 1, H, dk, dv)
    names = ("q", "k", "v", "dO")
    clean = dict(zip(names, (q, k, v, dO)))

    def run(t):
        o, S = block.linattn_forward(t["q"], t["k"], t["v"], lg, state=st)
        d = block.linattn_backward(t["q"], t["k"], t["v"], lg, t["dO"], state=st, dstate_out=ds)
        return {"o": o, "S": S, **{"d" + n: d[n] for n in "qkv"}, "dS": d["state"]}

    want = run(clean)
    assert all(torch.isfinite(t).all() for t in want.values())
    before, after, own, others = (lambda s: slice(0, s)), (lambda s: slice(s + 1, T)), "own", "all"
    # rows that a value of each input's token s does not reach
    untouched = {
        "q": {"o": own, "S": others, "dq": others, "dk": after, "dv": after},
        "k": {"o": before, "dq": before, "dk": others, "dv": own, "dS": others},
        "v": {"o": before, "dq": before, "dk": own, "dv": others, "dS": others},
        "dO": {"o": others, "S": others, "dq": own, "dk": after, "dv": after},
    }
    for s in sorted({0, 1, T // 2, T - 1}):
        for name in names:
            t = dict(clean)
            t[name] = clean[name].clone()
            t[name][0, s, 0, 5] = bad
            got = run(t)
            say(T, dtype, bad, s, name)
            for out, rows in untouched[name].items():
                a, b = got[out], want[out]
                if rows == own:
                    keep = [i for i in range(T) if i != s]
                    a, b = a[:, keep], b[:, keep]
                elif rows != others:
                    a, b = a[:, rows(s)], b[:, rows(s)]
                assert torch.equal(a, b), (name, s, out)
            if name == "v":  # one value of v is one column of o
                keep = [c for c in range(dv) if c != 5]
                assert torch.equal(got["o"][..., keep], want["o"][..., keep])
                assert not torch.isfinite(got["o"][0, s:s + 8, 0, 5]).any()
            if name == "k":
                assert not torch.isfinite(got["o"][0, s:s + 8, 0]).any()
            if name == "dO":
                assert not torch.isfinite(got["dv"][0, max(0, s - 7):s + 1, 0, 5]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [29, 70, 1100])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 64), (1, 128), (2, 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_attention_infinities_square_heads(bad, G, d, T, dtype):
    """The same where keys and values are of one size, whose gradients of k and v come from one
    launch, with their own heads and shared ones, in one segment and in many."""
    H = 2
    g, q, k, v, _, st = attn_inputs(1, T, H, G, d, d, dtype, T + G)
    lg = torch.tensor([-1e-3, -0.5], device="cuda")
    dO, ds = normal(g, 1, T, H, d, dtype=dtype), normal(g, 1, H, d, d)
    clean = {"q": q, "k": k, "v": v, "dO": dO}

    def run(t):
        o, S = block.linattn_forward(t["q"], t["k"], t["v"], lg, state=st)
        x = block.linattn_backward(t["q"], t["k"], t["v"], lg, t["dO"], state=st, dstate_out=ds)
        return {"o": o, "S": S, **{"d" + n: x[n] for n in "qkv"}, "dS": x["state"]}

    want = run(clean)
    assert all(torch.isfinite(t).all() for t in want.values())
    for s in (0, T // 2, T - 1):
        own = [t for t in range(T) if t != s]
        before, after, every = list(range(s)), list(range(s + 1, T)), list(range(T))
        untouched = {
            "q": {"o": own, "S": None, "dq": every, "dk": after, "dv": after},
            "k": {"o": before, "dq": before, "dk": every, "dv": own, "dS": None},
            "v": {"o": before, "dq": before, "dk": own, "dv": every, "dS": None},
            "dO": {"o": every, "S": None, "dq": own, "dk": after, "dv": after},
        }
        for name in clean:
            t = dict(clean)
            t[name] = clean[name].clone()
            t[name][0, s, 0, 5] = bad
            got = run(t)
            say(T, G, d, dtype, bad, s, name)
            for out, rows in untouched[name].items():
                a, b = (got[out], want[out]) if rows is None else (got[out][:, rows], want[out][:, rows])
                assert torch.equal(a, b), (name, s, out)
            near = slice(max(0, s - 7), s + 1)
            if name == "q":
                assert not torch.isfinite(got["dk"][0, near, 0, 5]).any()
            if name == "dO":
                keep = [c for c in range(d) if c != 5]
                assert torch.equal(got["dv"][..., keep], want["dv"][..., keep])
                assert not torch.isfinite(got["dv"][0, near, 0, 5]).any()
            if name == "v":
                assert not torch.isfinite(got["dk"][0, s, 0]).any()
                assert not torch.isfinite(got["o"][0, s:s + 8, 0, 5]).any()


# What three bf16 terms a weighted value keep, the 24 bits of fp32, is lost only by the
# fp32 sums: the weight, its product, six accumulations of a chunk and the decay, each
# within 2^-24 (rms 2^-24 / sqrt 3), 1.6 * 2^-24 a chunk; over the n chunks that a state
# remembers the roundings add like sqrt n.  Up to 35 chunks here: 10 * 2^-24, bound 2^-20
# (two terms: 2^-18 a value).
TOL_STATE_SUMS = 2.0 ** -20


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,H,G,d", [(1, 1100, 2, 2, 64), (2, 1100, 2, 1, 64), (1, 1100, 2, 2, 128),
                                       (1, 1100, 2, 1, 128), (1, 777, 4, 2, 104)])
def test_attention_gradients_of_many_segments(B, T, H, G, d, dtype, ragged):
    """More than eight segments, whose states a launch of its own adds up, for both directions at
    once: against the 64-bit form, and the states as exact as fp32 sums."""
    say(B, T, H, G, d, dtype, ragged)
    g, q, k, v, lg, st = attn_inputs(B, T, H, G, d, d, dtype, T + d)
    lg[0] = -1e-3
    dO, ds = normal(g, B, T, H, d, dtype=dtype), normal(g, B, H, d, d)
    lens = [T - 61, 643][:B] if ragged else None
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, S = block.linattn_forward(q, k, v, lg, scale=0.3, state=st, lengths=ln)
    got = block.linattn_backward(q, k, v, lg, dO, scale=0.3, state=st, dstate_out=ds, lengths=ln)
    o64, S64 = ref.linattn(f64(q), f64(k), f64(v), f64(lg), 0.3, f64(st), lens)
    want = ref.linattn_grads(f64(q), f64(k), f64(v), f64(lg), 0.3, f64(dO), f64(st), f64(ds), lens)
    err = {"o": rel(f64(o), o64), **{n: rel(f64(got[n]), w) for n, w in zip("qkv", want)}}
    states = rel(f64(S), S64), rel(f64(got["state"]), want[3])
    say("  ", {n: "%.2e" % e for n, e in err.items()}, "states %.2e %.2e" % states)
    assert all(e <= TOL_CHUNK[dtype] for e in err.values())
    assert max(states) <= TOL_STATE_SUMS


# Each of some hundred segments' sums is good to 2^-22 (eight chunks, see above); adding n of
# them up rounds the sum n times, 2^-24 / sqrt 3 rms each, of a sum that grows: sqrt(n / 2)
# of them, 9 * 2^-24 for 512 segments, 10 with the segments' own; bound twice that.
TOL_STATE_LONG = 2.0 ** -19.5


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_states_that_remember_many_segments(dtype):
    """131072 tokens with memories of 33000 and a million: the segments' factor is applied some
    hundred times, so that its own rounding (3e-8) must not be applied with it."""
    T, H, d = 131072, 2, 64
    g = gen(16)
    q, k, v, dO = (normal(g, 1, T, H, d, dtype=dtype) for _ in range(4))
    lg = torch.tensor([-1e-6, -3e-5], device="cuda")
    _, S = block.linattn_forward(q, k, v, lg)
    got = block.linattn_backward(q, k, v, lg, dO, scale=1.0, state=torch.zeros_like(S))
    for h in range(H):
        t = torch.arange(T, dtype=torch.float64)
        w = torch.exp(float(lg[h]) * t)[:, None]
        kh, vh, qh, dh = (x[0, :, h].cpu().double() for x in (k, v, q, dO))
        err = (rel(f64(S[0, h]), (kh * w.flip(0)).t() @ vh),
               rel(f64(got["state"][0, h]), (qh * w * np.exp(float(lg[h]))).t() @ dh))
        say(dtype, float(lg[h]), "%.2e %.2e" % err)
        assert max(err) <= TOL_STATE_LONG


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 4])
def test_attention_sessions_of_many_tokens(T, dtype):
    """A state of size 1 carried through 4000 tokens, T at a call, that add 0.6 to it: each token
    rounds it (the product's rest, the sum: 2 * 2^-24 / sqrt 3 rms), independently as what is added
    differs: sqrt(4000) of them, 73 * 2^-24, bound 2^-17.  The rounding of the decay itself (up
    to 2^-25) must not be among what is repeated: 4000 * 2^-25 is 1.2e-4."""
    H, d, n = 4, 64, 4000
    g = gen(18)
    q, k, v = (normal(g, 1, n, H, d, dtype=dtype, std=s) for s in (1.0, 0.01, 1.0))
    lg = torch.tensor([-2e-6, -7e-6, -3e-5, -3e-4], device="cuda")
    st = normal(g, 1, H, d, d)
    S = st.clone()
    for t in range(0, n, T):
        c = slice(t, t + T)
        o, _ = block.linattn_forward(q[:, c], k[:, c], v[:, c], lg, state=S, state_out=S)
    t = torch.arange(n, dtype=torch.float64)
    for h in range(H):
        w = torch.exp(float(lg[h]) * (n - 1 - t))[:, None]
        kh, vh = (x[0, :, h].cpu().double() for x in (k, v))
        want = st[0, h].cpu().double() * np.exp(float(lg[h]) * n) + (kh * w).t() @ vh
        e = rel(f64(S[0, h]), want)
        say(T, dtype, float(lg[h]), "%.2e" % e)
        assert e <= 2.0 ** -17
        assert rel(f64(o[0, -1, h]), q[0, -1, h].cpu().double() @ want * d ** -0.5) <= TOL_ROUND[dtype] + 2.0 ** -17


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 8, 32, 33, 70])
def test_attention_sessions_in_pieces(T, dtype):
    """The same in calls of the chunked form: each rounds the state some eight times (six
    accumulations and two decays a chunk), 1.6 * 2^-24 rms, sqrt(4000 / 5) of them: 46 * 2^-24,
    bound 2^-17.4.  The rounding of a last chunk's decay, or of a call's first one, up to 2^-24
    for each call, must not be among what is repeated: 4.8e-5 for 800 calls."""
    H, d, n = 4, 64, 4000
    g = gen(19)
    q, k, v = (normal(g, 1, n, H, d, dtype=dtype, std=s) for s in (1.0, 0.01, 1.0))
    lg = torch.tensor([-2e-6, -7e-6, -3e-5, -1e-4], device="cuda")
    st = normal(g, 1, H, d, d)
    S = st.clone()
    for t in range(0, n, T):
        c = slice(t, min(t + T, n))
        block.linattn_forward(q[:, c], k[:, c], v[:, c], lg, state=S, state_out=S)
    t = torch.arange(n, dtype=torch.float64)
    for h in range(H):
        w = torch.exp(float(lg[h]) * (n - 1 - t))[:, None]
        kh, vh = (x[0, :, h].cpu().double() for x in (k, v))
        want = st[0, h].cpu().double() * np.exp(float(lg[h]) * n) + (kh * w).t() @ vh
        e = rel(f64(S[0, h]), want)
        say(T, dtype, float(lg[h]), "%.2e" % e)
        assert e <= 2.0 ** -17.4


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_sessions_in_calls_of_few_segments(dtype):
    """The same in 128 calls of 512 tokens, each in eight segments: 2048 chunks of 1.6 * 2^-24 rms,
    of a state that what is added makes four times larger: sqrt(2048 / 2) of them, 51 * 2^-24,
    bound 2^-18.  The segments' factors, rounded by 2.7e-8 to 3e-8 for these decays, must not
    be repeated 1024 times with their rounding: 3e-5."""
    H, d, T, n = 4, 64, 512, 65536
    g = gen(20)
    q, k, v = (normal(g, 1, n, H, d, dtype=dtype, std=s) for s in (1.0, 0.015, 1.0))
    lg = torch.tensor([-1.5e-6, -5.5e-6, -7e-6, -1.05e-5], device="cuda")
    st = normal(g, 1, H, d, d)
    S = st.clone()
    for t in range(0, n, T):
        c = slice(t, t + T)
        block.linattn_forward(q[:, c], k[:, c], v[:, c], lg, state=S, state_out=S)
    t = torch.arange(n, dtype=torch.float64)
    for h in range(H):
        w = torch.exp(float(lg[h]) * (n - 1 - t))[:, None]
        kh, vh = (x[0, :, h].cpu().double() for x in (k, v))
        want = st[0, h].cpu().double() * np.exp(float(lg[h]) * n) + (kh * w).t() @ vh
        e = rel(f64(S[0, h]), want)
        say(dtype, float(lg[h]), "%.2e" % e)
        assert e <= 2.0 ** -18


@pytest.mark.parametrize("T", [4, 70, 600])
def test_attention_layouts(T):
    """Head-first storage, slices of one projection, a batch repeated by a stride of 0: as
    contiguous copies, bit for bit."""
    B, H, G, dk, dv = 2, 4, 2, 64, 72
    g = gen(T)
    lg = -torch.rand(H, generator=g).cuda() * 0.1
    st = normal(g, B, H, dk, dv)
    fused = normal(g, B, T, H * dk + G * dk + G * dv, dtype=BF16)
    q = fused[..., :H * dk].unflatten(-1, (H, dk))
    k = fused[..., H * dk:(H + G) * dk].unflatten(-1, (G, dk))
    v = fused[..., (H + G) * dk:].unflatten(-1, (G, dv))
    heads_first = [normal(g, B, n, T, d, dtype=BF16).transpose(1, 2)
                   for n, d in ((H, dk), (G, dk), (G, dv))]
    tokens_first = [normal(g, T, B, n, d, dtype=BF16).transpose(0, 1)
                    for n, d in ((H, dk), (G, dk), (G, dv))]
    repeated = [t[:1].expand(B, -1, -1, -1) for t in (q, k, v)]
    dO = normal(g, B, H, T, dv, dtype=BF16).transpose(1, 2)
    for qkv in ((q, k, v), heads_first, tokens_first, repeated):
        plain = [t.contiguous() for t in qkv]
        o, S = block.linattn_forward(*qkv, lg, state=st)
        o0, S0 = block.linattn_forward(*plain, lg, state=st)
        assert torch.equal(o, o0) and torch.equal(S, S0)
        a = block.linattn_backward(*qkv, lg, dO, state=st)
        b = block.linattn_backward(*plain, lg, dO.contiguous(), state=st)
        assert all(torch.equal(a[n], b[n]) for n in a)
    # o in a layout of its own
    out = torch.full((B, H, T, dv + 8), 5.0, dtype=BF16, device="cuda")
    o0, _ = block.linattn_forward(q, k, v, lg, state=st)
    desc = block.make_linattn_desc(B, T, H, G, dk, dv, BF16, dk ** -0.5, q.stride()[:3],
                                   k.stride()[:3], v.stride()[:3],
                                   (H * T * (dv + 8), dv + 8, T * (dv + 8)))
    ws = torch.empty(block.ttt_linattn_workspace_size(desc) or 1, dtype=torch.uint8, device="cuda")
    block.ttt_linattn_forward(desc, q, k, v, lg, None, st, None, out, ws)
    assert torch.equal(out[..., :dv].transpose(1, 2), o0) and (out[..., dv:] == 5.0).all()


def test_attention_offsets_past_32_bits():
    # tokens 2^26 values apart: the last of 70 is 4.6e9 values from the first
    T, d, far = 70, 64, 1 << 26
    big = torch.empty(T * far, dtype=BF16, device="cuda").view(T, far)
    g = gen(4)
    for at, n in ((0, 3 * d), (far - d, d)):
        big[:, at:at + n] = normal(g, T, n, dtype=BF16)
    q, k, v, dO = (big[None, :, None, at:at + d] for at in (0, d, 2 * d, far - d))
    lg = torch.tensor([-0.05], device="cuda")
    c = [t.contiguous() for t in (q, k, v, dO)]
    o, S = block.linattn_forward(q, k, v, lg)
    o0, S0 = block.linattn_forward(*c[:3], lg)
    assert torch.equal(o, o0) and torch.equal(S, S0)
    a, b = block.linattn_backward(q, k, v, lg, dO), block.linattn_backward(*c[:3], lg, c[3])
    assert all(torch.equal(a[n], b[n]) for n in "qkv")
    o, _ = block.linattn_forward(q[:, -4:], k[:, -4:], v[:, -4:], lg)
    assert torch.equal(o, block.linattn_forward(*(t[:, -4:].contiguous() for t in c[:3]), lg)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dv", [64, 128])
def test_attention_one_token_with_a_far_stride(dv, dtype):
    """The stride between the tokens of one token means nothing, whatever it is: the same results,
    bit for bit."""
    B, H, G, dk = 3, 4, 2, 64
    g, q, k, v, lg, st = attn_inputs(B, 1, H, G, dk, dv, dtype, 14)
    dO, ds = normal(g, B, 1, H, dv, dtype=dtype), normal(g, B, H, dk, dv)
    want = block.linattn_backward(q, k, v, lg, dO, scale=0.3, state=st, dstate_out=ds)
    want_o, _ = block.linattn_forward(q, k, v, lg, scale=0.3, state=st)
    new = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    for far in (0, 1 << 27, 1 << 30, 1 << 40):
        say(dv, dtype, far)
        desc = block.make_linattn_desc(B, 1, H, G, dk, dv, dtype, 0.3, (H * dk, far, dk),
                                       (G * dk, far, dk), (G * dv, far, dv), (H * dv, far, dv))
        ws = torch.empty(block.ttt_linattn_backward_workspace_size(desc) or 1, dtype=torch.uint8,
                         device="cuda")
        got = {"q": new(q), "k": new(k), "v": new(v), "state": new(st)}
        block.ttt_linattn_backward(desc, q, k, v, lg, None, st, dO, ds, *got.values(), ws)
        assert all(torch.equal(got[n], want[n]) for n in got)
        o = new(want_o)
        block.ttt_linattn_forward(desc, q, k, v, lg, None, st, None, o)
        assert torch.equal(o, want_o)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_prompt_then_tokens(dtype):
    """A prompt in pieces and single tokens continue one state."""
    B, T, H, G, dk, dv = 2, 300, 4, 2, 64, 64
    _, q, k, v, lg, _ = attn_inputs(B, T, H, G, dk, dv, dtype, 21)
    o64, S64 = ref.linattn(f64(q), f64(k), f64(v), f64(lg), dk ** -0.5)
    st, parts, p = None, [], 0
    for n in (200, 40, 9, 8, 1, 1, 3, 38):
        s = slice(p, p + n)
        o, st = block.linattn_forward(q[:, s], k[:, s], v[:, s], lg, state=st, state_out=st)
        parts.append(o)
        p += n
    assert p == T
    assert rel(f64(torch.cat(parts, 1)), o64) <= TOL_CHUNK[dtype]
    assert rel(f64(st), S64) <= TOL_STATE[dtype]


def test_another_stream():
    g, q, k, v, lg, st = attn_inputs(2, 600, 4, 4, 64, 64, BF16, 2)
    x, w = normal(g, 64, 2560, dtype=BF16), normal(g, 2560, dtype=BF16)
    o, S = block.linattn_forward(q, k, v, lg, state=st)
    y, _, _ = block.add_rmsnorm(x, None, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):  # the binding follows the current stream
        o1, S1 = block.linattn_forward(q, k, v, lg, state=st)
        y1, _, _ = block.add_rmsnorm(x, None, w)
    s.synchronize()
    assert torch.equal(o1, o) and torch.equal(S1, S) and torch.equal(y1, y)


def test_stream_argument_owns_its_allocations():
    """stream=s: what the call allocates belongs to s, so that allocations of the stream around
    it, filled at once, cannot land in memory that s still works on."""
    g, q, k, v, lg, st = attn_inputs(1, 6000, 4, 4, 64, 64, BF16, 12)
    dO = normal(g, 1, 6000, 4, 64, dtype=BF16)
    r, w = normal(g, 4096, 2560, dtype=BF16), normal(g, 2560, dtype=BF16)
    calls = (lambda **kw: block.linattn_forward(q, k, v, lg, state=st, **kw),
             lambda **kw: tuple(block.linattn_backward(q, k, v, lg, dO, state=st, **kw).values()),
             lambda **kw: block.add_rmsnorm_backward(r, r, w, **kw),
             lambda **kw: block.add_rmsnorm(r, r, w, **kw)[:2])
    s = torch.cuda.Stream()
    busy = torch.ones(1 << 26, device="cuda")
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        for stream in (s, s.cuda_stream):
            with torch.cuda.stream(s):
                busy.mul_(1.0)  # s is behind the current stream
            got = call(stream=stream)
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                    for n in (1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            del junk, got


def test_null_stream_argument():
    """stream=0, as the default stream's handle is: behind what is pending there, and in front of
    what follows."""
    g, q, k, v, lg, st = attn_inputs(1, 700, 4, 4, 64, 64, BF16, 13)
    dO = normal(g, 1, 700, 4, 64, dtype=BF16)
    x, w = normal(g, 512, 2560, dtype=BF16), normal(g, 2560, dtype=BF16)
    assert torch.cuda.current_stream().cuda_stream == torch.cuda.default_stream().cuda_stream == 0
    with block._on(0, q):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    calls = ((lambda q, x, **kw: block.linattn_forward(q, k, v, lg, state=st, **kw)),
             (lambda q, x, **kw: tuple(block.linattn_backward(q, k, v, lg, dO, state=st, **kw).values())),
             (lambda q, x, **kw: block.add_rmsnorm_backward(x, x, w, **kw)),
             (lambda q, x, **kw: block.add_rmsnorm(x, x, w, **kw)[:2]))
    busy = torch.ones(1 << 26, device="cuda")
    for call in calls:
        want = [t.clone() for t in call(q, x)]
        torch.cuda.synchronize()
        for stream in (0, torch.cuda.default_stream()):
            q2, x2 = torch.zeros_like(q), torch.zeros_like(x)
            torch.cuda.synchronize()
            for _ in range(20):
                busy.mul_(1.0)
            q2.copy_(q)
            x2.copy_(x)
            got = [t.clone() for t in call(q2, x2, stream=stream)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays_equal_eager():
    g, q, k, v, lg, st = attn_inputs(1, 700, 4, 2, 64, 64, BF16, 3)
    dO = normal(g, 1, 700, 4, 64, dtype=BF16)
    x, w = normal(g, 300, 1024, dtype=BF16), normal(g, 1024, dtype=BF16)
    desc = block.make_linattn_desc(1, 700, 4, 2, 64, 64, BF16, 0.125)
    nd = block.make_addnorm_desc(300, 1024, BF16)
    new = lambda t: torch.empty(t.shape, dtype=t.dtype, device="cuda")  # noqa: E731
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    ws, wb = (byte(f(desc) or 1) for f in (block.ttt_linattn_workspace_size,
                                           block.ttt_linattn_backward_workspace_size))
    wn = byte(block.ttt_addnorm_backward_workspace_size(nd))
    o, S, dq, dk, dv, dS = new(dO), new(st), new(q), new(k), new(v), new(st)
    one, So = new(dO[:, :1]), new(st)
    y, r, dr, dw = new(x), new(x), new(x), torch.empty(1024, device="cuda")
    d1 = block.make_linattn_desc(1, 1, 4, 2, 64, 64, BF16, 0.125)

    def calls(stream=None):
        block.ttt_linattn_forward(desc, q, k, v, lg, None, st, S, o, ws, stream=stream)
        block.ttt_linattn_forward(d1, q, k, v, lg, None, st, So, one, stream=stream)
        block.ttt_linattn_backward(desc, q, k, v, lg, None, st, dO, S, dq, dk, dv, dS, wb,
                                   stream=stream)
        block.ttt_addnorm_forward(nd, x, x, w, r, y, stream=stream)
        block.ttt_addnorm_backward(nd, y, r, w, None, dr, None, dw, wn, stream=stream)

    calls()
    torch.cuda.synchronize()
    outs = [o, S, one, So, dq, dk, dv, dS, y, r, dr, dw]
    refs = [t.clone() for t in outs]
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            calls(s)
    scratch = torch.ones(1 << 20, device="cuda")
    for i in range(3):
        scratch.mul_(1.5).add_(i)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, refs)), i
