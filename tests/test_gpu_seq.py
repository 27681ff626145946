"""The sequence operators on the GPU against their 64-bit forms: the embedding and
its gradient, the gated linear recurrence with its gradients, activations in 8
bits and the weight gradient from them, at the sizes, strides, masks and values
where they can go wrong.

Tolerances (relative Frobenius), from the number formats:
  fp32: each result is a sum of products with relative rounding 2^-24 a term, at
        most some hundred of them one after the other: 2e-6 (2^-24 times 32);
  bf16 result of fp32 arithmetic: one rounding, at most 2^-8 a value: 2^-8.
The lookup rounds one fp32 product, the 8-bit codes one exact quotient: both are
compared bit by bit.
"""
import numpy as np
import pytest
import torch

from chunk_wise_weight_chunked_amd import seq
from chunk_wise_weight_chunked_amd import ttt_mlp as tm

import _seq_ref as ref
from _block_ref import f64, rel

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TOL_F32 = 2e-6
TOL = {F32: TOL_F32, BF16: 2.0 ** -8}


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


# ---------------------------------------------------------------- embedding
def some_ids(g, N, V, dtype, hot=0.3):
    """Ids of which a part is one and the same, some outside the table."""
    ids = torch.randint(0, V, (N,), generator=g)
    ids[torch.rand(N, generator=g) < hot] = V // 2
    odd = torch.rand(N, generator=g)
    ids[odd < 0.02] = -1
    ids[(odd >= 0.02) & (odd < 0.04)] = V
    if dtype == torch.int64:
        ids[(odd >= 0.04) & (odd < 0.05)] = (1 << 32) + 1
    return ids.to(dtype)


@pytest.mark.parametrize("id_dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("N,V,d", [(1, 1, 8), (5, 7, 64), (33, 100, 128), (70, 50, 136),
                                   (300, 1000, 200), (9, 40, 2560), (1000, 33, 1000)])
def test_embed_forward(N, V, d, dtype, out, id_dtype):
    say(N, V, d, dtype, out, id_dtype)
    g = gen(N + d)
    table, ids = normal(g, V, d, dtype=dtype), some_ids(g, N, V, id_dtype)
    got = seq.embed_forward(ids.cuda(), table, 1.7, out_dtype=out)
    ok = (ids >= 0) & (ids < V)
    want = table.cpu().float()[ids.long().clamp(0, V - 1)] * torch.tensor(1.7)
    want = torch.where(ok[:, None], want, 0.0).to(out)
    assert got.dtype == out and torch.equal(got.cpu(), want)


def test_embed_forward_shapes_and_values():
    g = gen(1)
    table = normal(g, 20, 64, dtype=BF16)
    table[3, 5] = float("inf")
    table[4, 6] = float("nan")
    table[0] = float("nan")  # the row an id outside must not bring in
    ids = torch.tensor([[3, 4, -1], [25, 1, 1]]).cuda()
    got = seq.embed_forward(ids, table)
    assert got.shape == (2, 3, 64)
    assert torch.isinf(got[0, 0, 5]) and torch.isnan(got[0, 1, 6])
    assert (got[0, 2] == 0).all() and (got[1, 0] == 0).all()
    assert torch.equal(got[1, 1], table[1]) and torch.equal(got[1, 2], table[1])
    assert seq.embed_forward(torch.tensor(7).cuda(), table).shape == (64,)


# tokens, vocabulary, columns: one piece of the sorted tokens and many, one tile of the
# sort and many, one digit and two, columns of a wave and more
EMBED_SHAPES = [(1, 1, 8), (3, 1, 64), (31, 5, 64), (32, 5, 128), (33, 2, 136), (64, 64, 200),
                (500, 600, 520), (700, 3, 1000), (4096, 300, 64), (4097, 511, 72), (9000, 512, 64),
                (9000, 40000, 72), (20000, 7, 40), (300, 131072, 64), (513, 50, 2560),
                (6144, 700, 24), (6145, 700, 24), (8192, 700, 24), (8193, 700, 24),
                (9000, 300000, 8), (700, 1 << 20, 8),
                (20, 1000, 2560), (64, 3, 1032), (65, 64, 200), (128, 3, 1032), (129, 64, 200),
                (128, 300000, 8), (2, 1 << 20, 8), (20480, 90, 8), (20481, 90, 8), (2100, 50, 2056)]


@pytest.mark.parametrize("dtype,gd", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("N,V,d", EMBED_SHAPES)
def test_embed_backward(N, V, d, dtype, gd):
    say(N, V, d, dtype, gd)
    g = gen(N + V)
    for id_dtype in (torch.int64, torch.int32):
        ids = some_ids(g, N, V, id_dtype)
        dout = normal(g, N, d, dtype=dtype)
        bad = (ids < 0) | (ids >= V)
        dout[bad.cuda()] = float("nan")  # what has no row must not reach one
        clean = torch.where(bad[:, None], 0.0, dout.cpu().double()).numpy()
        got = seq.embed_backward(dout, ids.cuda(), V, 0.6, grad_dtype=gd)
        want = ref.embed_grad(clean, ids.numpy(), V, np.float64(np.float32(0.6)))
        e = rel(f64(got), want)
        say("  %.2e" % e)
        assert got.dtype == gd and e <= TOL[gd]
        none = np.setdiff1d(np.arange(V), ids.numpy())
        assert not got.cpu()[none].any()
        again = seq.embed_backward(dout, ids.cuda(), V, 0.6, grad_dtype=gd)
        assert torch.equal(again, got)
        # added to what is there; rows without tokens keep their bits
        start = normal(g, V, d, dtype=gd)
        start[none] = float("nan")
        keep = start.clone()
        grad = seq.embed_backward(dout, ids.cuda(), V, 0.6, grad=start)
        assert grad is start
        some = np.setdiff1d(np.arange(V), none)
        want = ref.embed_grad(clean, ids.numpy(), V, np.float64(np.float32(0.6)), f64(keep))
        if len(some):
            assert rel(f64(grad)[some], want[some]) <= TOL[gd]
        assert torch.isnan(grad[none]).all()


@pytest.mark.parametrize("lead", [0, 1, 31, 2047, 2048, 5000])
def test_embed_backward_ids_of_very_many_tokens(lead):
    """One id with nearly all tokens, begun anywhere in the sorted order, between rare ones."""
    N, V, d = 140000, 50, 24
    g = gen(lead)
    ids = torch.full((N,), 20)
    at = torch.randperm(N, generator=g)
    ids[at[:lead]] = torch.randint(0, 20, (lead,), generator=g)
    ids[at[lead:lead + 700]] = torch.randint(21, V, (700,), generator=g)
    dout = normal(g, N, d)
    want = ref.embed_grad(f64(dout), ids.numpy(), V, 1.0)
    got = f64(seq.embed_backward(dout, ids.cuda(), V))
    for v in range(V):
        if want[v].any():
            assert rel(got[v], want[v]) <= TOL_F32, v
    assert rel(got, want) <= TOL_F32
    start = normal(g, V, d)
    want = want + f64(start)
    assert rel(f64(seq.embed_backward(dout, ids.cuda(), V, grad=start)), want) <= TOL_F32


def test_embed_backward_is_the_forwards():
    """<dout, embed(table)> is linear in the table: its differences are the gradient."""
    g = gen(5)
    N, V, d = 800, 120, 72
    ids, dout = some_ids(g, N, V, torch.int64).cuda(), normal(g, N, d)
    u = normal(g, V, d)
    got = float((seq.embed_backward(dout, ids, V, 0.5).double() * u.double()).sum())
    diff = float((dout.double() * seq.embed_forward(ids, u, 0.5).double()).sum())
    assert abs(got - diff) <= TOL_F32 * float(dout.double().norm() * u.double().norm())


def test_embed_backward_infinities_stay_in_their_rows():
    g = gen(6)
    ids = torch.randint(0, 40, (300,), generator=g)
    dout = normal(g, 300, 64)
    dout[7, 3], dout[8, 4] = float("inf"), float("nan")
    got = seq.embed_backward(dout, ids.cuda(), 40).cpu()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[ids[7], 3] = want[ids[8], 4] = True
    assert torch.equal(bad, want)


# ----------------------------------------------------- gated linear recurrence
# (B, T, d): few tokens without tiles; one tile of up to 32, 64 or 128 tokens, many tiles; one
# strip of 64 channels, parts of one, several
REC_SHAPES = [(1, 1, 8), (3, 1, 200), (2, 5, 64), (2, 6, 72), (3, 7, 64), (1, 8, 72), (2, 9, 8),
              (1, 31, 64), (3, 32, 136), (2, 33, 64), (3, 64, 72), (1, 65, 8), (2, 100, 136),
              (1, 127, 64), (3, 128, 72), (1, 129, 8), (2, 257, 64), (1, 700, 200), (2, 1100, 64),
              (1, 4500, 72)]


def rec_inputs(B, T, d, dtype, seed, wide=False):
    g = gen(seed)
    if wide:  # slices of one projection's rows, between others
        p = normal(g, B, T, 4 * d, dtype=dtype)
        x, dg, ig = p[..., d:2 * d], p[..., 2 * d:3 * d], p[..., :d]
    else:
        x, dg, ig = (normal(g, B, T, d, dtype=dtype) for _ in range(3))
    rate = torch.exp(torch.rand(d, generator=g) * 8 - 6).cuda()  # memories of one to 400 tokens
    return g, x, dg, ig, rate, normal(g, B, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", REC_SHAPES, ids=str)
def test_gatedrec_forward(shape, dtype):
    say(shape, dtype)
    B, T, d = shape
    for wide in (False, True):
        _, x, dg, ig, rate, st = rec_inputs(*shape, dtype, T + d, wide)
        for state in (None, st):
            h, S, none = seq.gatedrec_forward(x, dg, ig, rate, state=state)
            h64, S64 = ref.gatedrec(f64(x), f64(dg), f64(ig), f64(rate), f64(state))
            eh, es = rel(f64(h), h64), rel(f64(S), S64)
            say("  h %.2e state %.2e" % (eh, es))
            assert none is None and h.dtype == dtype and eh <= TOL[dtype] and es <= TOL_F32
    # in place, with the states in front of the tiles, and without a state out
    keep = st.clone()
    h2, S2, saved = seq.gatedrec_forward(x, dg, ig, rate, state=keep, state_out=keep, save=True)
    assert S2 is keep and torch.equal(keep, S) and torch.equal(h2, h)
    assert saved.shape == (B, -(-T // 128), d) and torch.equal(saved[:, 0], st)
    for j in range(1, saved.shape[1]):
        part = ref.gatedrec(f64(x)[:, :128 * j], f64(dg), f64(ig), f64(rate), f64(st))[1]
        assert rel(f64(saved[:, j]), part) <= TOL_F32
        if j > 3:
            break
    real = lambda t: [0 if n == 1 else s for n, s in zip(t.shape, t.stride()[:2])]  # noqa: E731
    out = torch.full((B, T, 2 * d), 7.0, dtype=dtype, device="cuda")
    desc = seq.make_gatedrec_desc(B, T, d, dtype, real(x), real(dg), real(ig),
                                  (2 * T * d, 2 * d))
    ws = torch.empty(seq.ttt_gatedrec_workspace_size(desc) or 1, dtype=torch.uint8, device="cuda")
    seq.ttt_gatedrec_forward(desc, x, dg, ig, rate, None, st, None, out, None, ws)
    assert torch.equal(out[..., :d], h) and (out[..., d:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 40, 600])
def test_gatedrec_lengths(T, dtype):
    lens = [0, 1, T - 1, T, T + 5, -3, T // 2, 33, 128, 129]
    B, d = len(lens), 72
    g, x, dg, ig, rate, st = rec_inputs(B, T, d, dtype, T)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = ln.clamp(0, T)
    # what lies behind a sequence's end must not be read into anything
    behind = torch.arange(T, device="cuda")[None, :] >= n[:, None]
    for i, t in enumerate((x, dg, ig)):
        t[behind] = (float("nan"), float("inf"), torch.finfo(dtype).min)[i]
    clean = [f64(torch.where(behind[..., None], torch.zeros_like(t), t)) for t in (x, dg, ig)]
    dh, ds = normal(g, B, T, d, dtype=dtype), normal(g, B, d)
    dh[behind] = float("nan")
    dh64 = f64(torch.where(behind[..., None], torch.zeros_like(dh), dh))
    for state, dstate in ((None, None), (st, ds)):
        h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, state=state, lengths=ln, save=True)
        h64, S64 = ref.gatedrec(*clean, f64(rate), f64(state), lens)
        assert (h[behind] == 0).all()
        assert rel(f64(h), h64) <= TOL[dtype] and rel(f64(S), S64) <= TOL_F32
        got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=dstate, lengths=ln)
        want = ref.gatedrec_grads(*clean, f64(rate), dh64, f64(state), f64(dstate), lens)
        for name, w in zip(("x", "decay_gate", "input_gate"), want):
            assert (got[name][behind] == 0).all()
            assert rel(f64(got[name]), w) <= TOL[dtype], name
        assert rel(f64(got["rate"]), want[3]) <= TOL_F32
        assert rel(f64(got["state"]), want[4]) <= TOL_F32
        if state is not None:
            assert torch.equal(S[0], st[0]) and torch.equal(S[5], st[5])  # no tokens
            assert torch.equal(got["state"][0], ds[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [7, 16, 17, 33, 65])
def test_gatedrec_many_sequences(T, dtype):
    """More of them than workgroups fit the chip, of which some are looked at."""
    B, d = 1 << 17, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dg, ig, dh = (new(B, T, d).to(dtype) for _ in range(4))
    rate, st, ds = new(d).abs() + 0.05, new(B, d), new(B, d)
    ln = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, state=st, lengths=ln, save=True)
    got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=ds, lengths=ln)
    some = torch.cat([torch.arange(40), torch.randint(0, B, (100,), generator=gen(T)),
                      torch.arange(B - 40, B)]).cuda()
    lens = ln[some].tolist()
    a = [f64(t[some]) for t in (x, dg, ig)]
    h64, S64 = ref.gatedrec(*a, f64(rate), f64(st[some]), lens)
    assert rel(f64(h[some]), h64) <= TOL[dtype] and rel(f64(S[some]), S64) <= TOL_F32
    want = ref.gatedrec_grads(*a, f64(rate), f64(dh[some]), f64(st[some]), f64(ds[some]), lens)
    for name, w in zip(("x", "decay_gate", "input_gate"), want):
        assert rel(f64(got[name][some]), w) <= TOL[dtype], name
    assert rel(f64(got["state"][some]), want[4]) <= TOL_F32
    # the rest by calls of their own, and the rate's gradient as their sum
    drate = torch.zeros(d, dtype=torch.float64, device="cuda")
    for p in torch.arange(B, device="cuda").split(B // 4):
        own = [t[p].contiguous() for t in (x, dg, ig)]
        h2, S2, saved2 = seq.gatedrec_forward(*own, rate, state=st[p], lengths=ln[p], save=True)
        assert rel(f64(h2), f64(h[p])) <= TOL[dtype] and rel(f64(S2), f64(S[p])) <= TOL_F32
        own = seq.gatedrec_backward(*own, rate, dh[p], saved2, dstate_out=ds[p], lengths=ln[p])
        assert all(torch.equal(own[n], got[n][p]) for n in ("x", "decay_gate", "input_gate", "state"))
        drate += own["rate"].double()
    assert rel(f64(got["rate"]), f64(drate)) <= TOL_F32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", REC_SHAPES, ids=str)
def test_gatedrec_backward(shape, dtype):
    say(shape, dtype)
    B, T, d = shape
    for wide in (False, True):
        g, x, dg, ig, rate, st = rec_inputs(*shape, dtype, T + 2 * d, wide)
        dh, ds = normal(g, B, T, 2 * d, dtype=dtype)[..., d:], normal(g, B, d)
        for state, dstate in ((None, None), (st, ds)):
            _, _, saved = seq.gatedrec_forward(x, dg, ig, rate, state=state, save=True)
            got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=dstate)
            want = ref.gatedrec_grads(f64(x), f64(dg), f64(ig), f64(rate), f64(dh), f64(state),
                                      f64(dstate))
            names = ("x", "decay_gate", "input_gate", "rate", "state")
            err = {n: rel(f64(got[n]), w) for n, w in zip(names, want)}
            say("  " + " ".join("%s %.2e" % p for p in err.items()))
            for n in names[:3]:
                assert got[n].dtype == dtype and err[n] <= TOL[dtype], n
            assert err["rate"] <= TOL_F32 and err["state"] <= TOL_F32
            again = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=dstate)
            assert all(torch.equal(again[n], got[n]) for n in names)
    real = lambda t: [0 if n == 1 else s for n, s in zip(t.shape, t.stride()[:2])]  # noqa: E731
    desc = seq.make_gatedrec_desc(B, T, d, dtype, real(x), real(dg), real(ig), real(dh))
    ws = torch.empty(seq.ttt_gatedrec_backward_workspace_size(desc) or 1, dtype=torch.uint8,
                     device="cuda")
    o = {n: torch.empty_like(got[n]) for n in names}
    seq.ttt_gatedrec_backward(desc, x, dg, ig, rate, None, saved, dh, ds, o["x"], o["decay_gate"],
                              o["input_gate"], o["rate"], ds, ws)  # the state's gradient in place
    assert all(torch.equal(o[n], got[n]) for n in names[:4]) and torch.equal(ds, got["state"])


def test_gatedrec_backward_against_differences():
    g, x, dg, ig, rate, st = rec_inputs(2, 300, 64, F32, 9)
    dh, ds = normal(g, 2, 300, 64), normal(g, 2, 64)
    u = [normal(g, *t.shape) for t in (x, dg, ig, st)] + [rate * normal(g, 64)]
    _, _, saved = seq.gatedrec_forward(x, dg, ig, rate, state=st, save=True)
    got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=ds)

    def f(e):
        h, S, _ = seq.gatedrec_forward(x + e * u[0], dg + e * u[1], ig + e * u[2],
                                       rate + e * u[4], state=st + e * u[3])
        return float((dh.double() * h.double()).sum() + (ds.double() * S.double()).sum())

    e = 2.0 ** -7
    diff = (f(e) - f(-e)) / (2 * e)
    grads = [got[n] for n in ("x", "decay_gate", "input_gate", "state", "rate")]
    parts = [float((a.double() * b.double()).sum()) for a, b in zip(grads, u)]
    # third derivatives: e^2 = 6e-5; rounding 2^-24 / e = 8e-6, of sums of size |dh| |h|
    size = sum(float(a.double().norm() * b.double().norm()) for a, b in zip(grads, u))
    assert abs(diff - sum(parts)) <= 1e-4 * size


@pytest.mark.parametrize("T", [5, 300, 20000])
def test_gatedrec_long_memories(T):
    """The same gates at every token and a decay so near 1 that its rounding to fp32 would be a
    large part of its distance from 1: repeated T times it would show."""
    d = 64
    rate = torch.logspace(-7, -3, d).cuda()
    x = torch.ones(1, T, d, device="cuda")
    gate = torch.zeros(1, T, d, device="cuda")
    st = torch.full((1, d), 3.0, device="cuda")
    h, S, saved = seq.gatedrec_forward(x, gate, gate, rate, state=st, save=True)
    h64, S64 = ref.gatedrec(f64(x), f64(gate), f64(gate), f64(rate), f64(st))
    assert rel(f64(h), h64) <= TOL_F32 and rel(f64(S), S64) <= TOL_F32
    # the state alone, kept for T tokens
    zero = torch.zeros_like(x)
    _, S, _ = seq.gatedrec_forward(zero, gate, gate, rate, state=st)
    assert rel(f64(S), 3.0 * np.exp(-0.5 * T * f64(rate))) <= TOL_F32
    got = seq.gatedrec_backward(x, gate, gate, rate, x, saved)
    want = ref.gatedrec_grads(f64(x), f64(gate), f64(gate), f64(rate), f64(x), f64(st))
    for n, w in zip(("x", "decay_gate", "input_gate", "rate", "state"), want):
        assert rel(f64(got[n]), w) <= TOL_F32, n


@pytest.mark.parametrize("T", [6, 400])
def test_gatedrec_values_out_of_the_ordinary(T):
    d = 64
    g, x, dg, ig, rate, st = rec_inputs(1, T, d, F32, 2)
    inf = float("inf")
    rate[0] = 0.0             # nothing decays, nothing enters
    rate[1] = 1e30            # a = 0: h = i x
    rate[2] = -1.0            # not allowed: NaN
    dg[..., 3] = -inf         # sigmoid 0: as a rate of 0
    dg[..., 4] = inf          # sigmoid 1
    ig[..., 5] = -inf         # nothing enters
    ig[..., 6] = inf
    x[0, 2, 7] = inf          # its channel alone, from its token on
    dg[0, 3, 8] = float("nan")
    rate[9] = 1e-38           # a state kept for good
    clean = [t.clone() for t in (x, dg, ig, rate)]
    h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, state=st, save=True)
    assert torch.isnan(h[..., 2]).all()
    assert torch.isfinite(h[0, :2, 7]).all() and not torch.isfinite(h[0, 2, 7])
    assert torch.isfinite(h[0, :3, 8]).all() and torch.isnan(h[0, 3:, 8]).all()
    assert (h[..., 0] == st[:, :1]).all() and (h[..., 3] == st[:, 3:4]).all()
    fine = [c for c in range(d) if c not in (2, 7, 8)]
    h64, S64 = ref.gatedrec(*(f64(t)[..., fine] for t in (x, dg, ig, rate, st)))
    assert rel(f64(h)[..., fine], h64) <= TOL_F32
    dh, ds = normal(g, 1, T, d), normal(g, 1, d)
    got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=ds)
    want = ref.gatedrec_grads(*(f64(t)[..., fine] for t in (x, dg, ig, rate, dh, st, ds)))
    for n, w in zip(("x", "decay_gate", "input_gate", "rate", "state"), want):
        assert rel(f64(got[n])[..., fine], w) <= TOL_F32, n
    assert all(torch.equal(a, b) for a, b in zip(clean[:3], (x, dg, ig)) if a.isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 6, 40, 400])
def test_gatedrec_rates_of_minus_zero(T, dtype):
    """-0.0 (minus the logarithm of 1) is a rate of 0: the state and what comes from behind are
    kept, bit for bit as with 0.0."""
    B, d = 2, 72
    g, x, dg, ig, rate, st = rec_inputs(B, T, d, dtype, T)
    dh, ds = normal(g, B, T, d, dtype=dtype), normal(g, B, d)
    rate[::2] = 0.0
    minus = torch.where(rate == 0, -rate, rate)
    assert torch.signbit(minus[::2]).all()
    results = []
    for r in (rate, minus):
        h, S, saved = seq.gatedrec_forward(x, dg, ig, r, state=st, save=True)
        got = seq.gatedrec_backward(x, dg, ig, r, dh, saved, dstate_out=ds)
        results.append([h, S, saved, *got.values()])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    h, S, saved = results[1][:3]
    kept = [c for c in range(0, d, 2)]
    assert torch.equal(S[:, kept], st[:, kept])
    assert (h[..., kept] == st[:, None, kept].to(dtype)).all()
    assert (saved[..., kept] == st[:, None, kept]).all()
    want = ref.gatedrec_grads(*(f64(t) for t in (x, dg, ig, minus, dh, st, ds)))
    assert rel(f64(got["state"]), want[4]) <= TOL_F32
    assert rel(f64(got["rate"]), want[3]) <= TOL_F32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [6, 40, 400])
def test_gatedrec_input_gates_far_down(T, dtype):
    """An input gate counts for as long as its sigmoid is a normal number of fp32 (2^-126 at a gate
    of -87.3): a channel a gate, x and dh large enough for the results to be normal too."""
    gates = torch.tensor([-20.0, -40.0, -60.0, -64.0, -66.0, -67.0, -68.0, -70.0, -75.0, -80.0,
                          -84.0, -85.0, -86.0, -87.0, -50.0, -30.0])
    d = len(gates)
    g, x, dg, _, rate, _ = rec_inputs(2, T, d, dtype, T + 1)
    ig = gates.to(dtype).cuda().expand(2, T, d)
    x, dh = x * 2.0 ** 30, normal(g, 2, T, d, dtype=dtype, std=2.0 ** 30)
    h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, save=True)
    got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved)
    a = [f64(t) for t in (x, dg, ig, rate)]
    h64, S64 = ref.gatedrec(*a)
    want = ref.gatedrec_grads(*a, f64(dh))
    pairs = [("h", h, h64), ("state", S, S64)]
    pairs += [(n, got[n], w) for n, w in zip(("x", "decay_gate", "input_gate"), want)]
    for c, gate in enumerate(ig[0, 0].tolist()):
        # e^-gate is 2 to a product of the gate and log2 e, which are rounded by 2^-24 and 2^-26
        # of it: as much of the exponent is off.  ddecay is the difference of two such terms
        # that do not depend on each other: sqrt(2) of what one may be off.
        far = 1.25 * abs(gate) * 2.0 ** -24
        for n, t, w in pairs:
            e = rel(f64(t)[..., c], w[..., c])
            tol = (TOL_F32 if n == "state" else TOL[dtype]) + far
            assert e <= tol * (2 ** 0.5 if n == "decay_gate" else 1), (n, gate, e)


def test_gatedrec_in_pieces():
    """A sequence fed in calls of any lengths gives one call's outputs to rounding."""
    B, T, d = 2, 700, 136
    _, x, dg, ig, rate, st = rec_inputs(B, T, d, F32, 4)
    h, S, _ = seq.gatedrec_forward(x, dg, ig, rate, state=st)
    state, at, parts = st.clone(), 0, []
    for n in (1, 1, 5, 8, 9, 128, 300, 1, 247):
        y, _, _ = seq.gatedrec_forward(*(t[:, at:at + n] for t in (x, dg, ig)), rate, state=state,
                                       state_out=state)
        parts.append(y)
        at += n
    assert at == T
    assert rel(f64(torch.cat(parts, 1)), f64(h)) <= TOL_F32 and rel(f64(state), f64(S)) <= TOL_F32


def test_gatedrec_repeated_inputs():
    """Strides of 0: one token's gates for all, one sequence's x for all."""
    B, T, d = 3, 260, 64
    g = gen(8)
    x = normal(g, 1, T, d).expand(B, T, d)
    dg = normal(g, B, 1, d).expand(B, T, d)
    ig, rate = normal(g, B, T, d), torch.full((d,), 0.1, device="cuda")
    dh = normal(g, 1, 1, d).expand(B, T, d)
    h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, save=True)
    full = [t.contiguous() for t in (x, dg, ig, dh)]
    h2, S2, saved2 = seq.gatedrec_forward(*full[:3], rate, save=True)
    assert torch.equal(h, h2) and torch.equal(S, S2) and torch.equal(saved, saved2)
    a = seq.gatedrec_backward(x, dg, ig, rate, dh, saved)
    b = seq.gatedrec_backward(*full[:3], rate, full[3], saved)
    assert all(torch.equal(a[n], b[n]) for n in a)


# ---------------------------------------------------------- activations in 8 bits
ACT_SHAPES = [(1, 8), (3, 24), (5, 32), (40, 40), (17, 128), (9, 136), (300, 200), (33, 1000),
              (6, 2560), (2, 4104)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", ACT_SHAPES)
def test_act8(rows, d, dtype):
    say(rows, d, dtype)
    g = gen(rows + d)
    x = (torch.randn((rows, d), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g)))
    x[0, :8] = 0
    x = x.to(dtype).cuda()
    codes, exps = seq.act8_store(x)
    wc, we = ref.act8(f64(x))
    assert np.array_equal(codes.cpu().numpy(), wc) and np.array_equal(exps.cpu().numpy(), we)
    for to in (BF16, F32):
        y = seq.act8_load(codes, exps, to)
        assert y.dtype == to and np.array_equal(f64(y), ref.act8_value(wc, we))
    wide = torch.full((rows, d + 24), 5.0, dtype=dtype, device="cuda")
    wide[:, 8:8 + d] = x
    c2, e2 = seq.act8_store(wide[:, 8:8 + d])
    assert torch.equal(c2, codes) and torch.equal(e2, exps)
    desc = seq.make_act8_desc(rows, d, dtype, d + 24)
    seq.ttt_act8_load(desc, codes, exps, wide[:, 8:8 + d])
    assert torch.equal(wide[:, 8:8 + d], seq.act8_load(codes, exps, dtype))
    assert (wide[:, :8] == 5).all() and (wide[:, 8 + d:] == 5).all()


def test_act8_values():
    """Largest values at, just below and just above what a scale holds, the smallest and largest
    numbers, ties, and groups that are not finite."""
    tops = []
    for e in (-149, -140, -133, -132, -126, -119, -20, 0, 1, 100, 120, 121):
        for m in (126.5, 127.0, 127.00001, 127.5, 128.0, 64.0, 63.5, 1.0):
            with np.errstate(over="ignore"):
                v = np.float32(m * 2.0 ** e)
            if np.isfinite(v):
                tops.append(v)
    tops += [np.float32(0), np.finfo(np.float32).max, np.float32(2.0 ** -149)]
    x = np.zeros((len(tops), 64), np.float32)
    for i, t in enumerate(tops):
        x[i, 0], x[i, 1] = t, -t
        x[i, 2:32] = t * np.linspace(-1, 1, 30, dtype=np.float32)
        x[i, 32:] = (np.arange(32) - 16 + 0.5) * np.float32(2.0 ** -3)  # ties: scale 1/8
    x = torch.from_numpy(x).cuda()
    codes, exps = seq.act8_store(x)
    wc, we = ref.act8(f64(x))
    assert np.array_equal(exps.cpu().numpy(), we) and np.array_equal(codes.cpu().numpy(), wc)
    y = seq.act8_load(codes, exps, F32)
    off = np.abs(f64(y) - f64(x))
    top = np.abs(f64(x)).reshape(len(tops), 2, 32).max(-1, keepdims=True)
    bound = np.maximum(top / 127, 2.0 ** -127)
    assert (off.reshape(len(tops), 2, 32) <= bound).all()
    x = torch.ones(4, 96, device="cuda")
    x[0, 3], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    for dt in (F32, BF16):
        codes, exps = seq.act8_store(x.to(dt))
        bad = torch.zeros(4, 3, dtype=torch.bool)
        bad[0, 0] = bad[1, 1] = bad[2, 2] = True
        assert torch.equal(exps.cpu() == 255, bad)
        for to in (F32, BF16):
            y = seq.act8_load(codes, exps, to).cpu()
            assert torch.equal(torch.isnan(y), bad.repeat_interleave(32, 1))
            assert (y[~torch.isnan(y)] == 1).all()


# rows, d_in, d_out: part of a tile, whole tiles, more than one, token slices
GRAD_SHAPES = [(1, 8, 8), (5, 40, 24), (64, 256, 256), (65, 264, 248), (300, 72, 520),
               (1000, 128, 328), (3001, 264, 72), (9000, 64, 64)]


@pytest.mark.parametrize("dtype,gd", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,d_in,d_out", GRAD_SHAPES)
def test_act8_weight_grad(rows, d_in, d_out, dtype, gd):
    say(rows, d_in, d_out, dtype, gd)
    g = gen(rows + d_out)
    codes, exps = seq.act8_store(normal(g, rows, d_in))
    wide = normal(g, rows, d_out + 16, dtype=dtype)
    x64 = ref.act8_value(codes.cpu().numpy(), exps.cpu().numpy())
    for dy in (wide[:, 8:8 + d_out].contiguous(), wide[:, 8:8 + d_out], wide[:, 16:]):
        want = x64.T @ f64(dy)
        got = seq.act8_weight_grad(codes, exps, dy, grad_dtype=gd)
        e = rel(f64(got), want)
        say("  %.2e" % e)
        assert got.shape == (d_in, d_out) and got.dtype == gd and e <= TOL[gd]
        assert torch.equal(seq.act8_weight_grad(codes, exps, dy, grad_dtype=gd), got)
    if gd == F32:
        start = normal(g, d_in, d_out, std=rows ** 0.5)
        keep = f64(start)
        grad = seq.act8_weight_grad(codes, exps, dy, grad=start)
        assert grad is start and rel(f64(grad), want + keep) <= TOL_F32


# wide tiles: whole ones and a rest in slices, slices alone; small tiles: whole ones, with a
# rest in slices, and more than one round of them
@pytest.mark.parametrize("rows,d_in,d_out,dtype,gd", [
    (8229, 2600, 6664, BF16, F32), (8229, 2600, 6664, BF16, BF16), (8229, 2600, 6664, F32, F32),
    (33001, 1032, 4104, BF16, F32), (17001, 1032, 4104, F32, F32), (130, 3000, 6000, BF16, F32),
    (700, 2568, 3336, F32, F32), (4000, 4104, 2056, BF16, F32),
    (700, 2568, 3336, BF16, F32), (700, 2568, 3336, BF16, BF16), (1100, 4104, 2056, BF16, F32)])
def test_act8_weight_grad_large(rows, d_in, d_out, dtype, gd):
    say(rows, d_in, d_out, dtype, gd)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    codes, exps = seq.act8_store(torch.randn(rows, d_in, generator=g, device="cuda"))
    wide = torch.randn(rows, d_out + 8, generator=g, device="cuda").to(dtype)
    dy = wide[:, 8:]
    x64 = seq.act8_load(codes, exps, F32).double()
    want = x64.t().contiguous() @ dy.double()
    got = seq.act8_weight_grad(codes, exps, dy, grad_dtype=gd)
    # against the norm of each row and column too, so that no tile hides behind the others
    off = got.double() - want
    for dim in (0, 1):
        e = float((off.norm(dim=dim) / want.norm(dim=dim)).max())
        say("  %.2e" % e)
        assert e <= TOL[gd]
    assert torch.equal(seq.act8_weight_grad(codes, exps, dy, grad_dtype=gd), got)
    if gd == F32:
        start = torch.randn(d_in, d_out, generator=g, device="cuda") * rows ** 0.5
        keep = start.double()
        seq.act8_weight_grad(codes, exps, dy, grad=start)
        assert float(((start.double() - keep - want).norm() / want.norm())) <= TOL_F32


@pytest.mark.parametrize("power", [-100, -115, -126, -130])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_act8_weight_grad_tiny(power, dtype):
    """Gradients near the end of the types' ranges: an fp32 dy counts in multiples of 2^-133."""
    g = gen(7)
    codes, exps = seq.act8_store(normal(g, 700, 256))
    dy = normal(g, 700, 264)
    dy = (dy.double() * 2.0 ** power).to(dtype)
    x64 = ref.act8_value(codes.cpu().numpy(), exps.cpu().numpy())
    want = x64.T @ f64(dy)
    got = f64(seq.act8_weight_grad(codes, exps, dy))
    # each of 700 additions may round to a multiple of 2^-149; dy's rest is below 2^-133
    lost = abs(x64).sum(0)[:, None] * 2.0 ** -133 if dtype == F32 else 0.0
    size = (want ** 2).mean() ** 0.5
    assert (abs(got - want) <= 8 * TOL_F32 * size + 3 * 700 * 2.0 ** -149 + lost).all()


def test_act8_weight_grad_rows_of_more_dimensions():
    g = gen(3)
    x, dy = normal(g, 3, 50, 64, dtype=BF16), normal(g, 3, 50, 40, dtype=BF16)
    codes, exps = seq.act8_store(x)
    assert codes.shape == (3, 50, 64) and exps.shape == (3, 50, 2)
    a = seq.act8_weight_grad(codes, exps, dy)
    b = seq.act8_weight_grad(codes.view(150, 64), exps.view(150, 2), dy.view(150, 40))
    assert torch.equal(a, b)
    want = f64(seq.act8_load(codes, exps)).reshape(150, 64).T @ f64(dy).reshape(150, 40)
    assert rel(f64(a), want) <= TOL_F32


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_act8_weight_grad_values_out_of_the_ordinary(dtype):
    """What is not finite reaches the row (a group of 32 input channels) or the column that the
    formula gives it to, and no other; dy at the ends of its type's range."""
    g = gen(12)
    rows, d_in, d_out = 200, 96, 64
    x, dy = normal(g, rows, d_in), normal(g, rows, d_out, dtype=dtype)
    x[5, 40] = float("nan")
    dy[7, 3], dy[8, 4] = float("inf"), float("nan")
    dy[:, 6] = torch.finfo(dtype).max
    dy[:, 7] *= 2.0 ** -100
    codes, exps = seq.act8_store(x)
    codes[:, 1] = 0
    codes[7, 2] = 0
    codes[3, 0], codes[4:, 0], codes[:3, 0] = 1, 0, 0  # one code alone: no overflow in column 6
    exps[:, 0] = 127
    got = f64(seq.act8_weight_grad(codes, exps, dy))
    bad = np.zeros((d_in, d_out), bool)
    bad[32:64] = True           # the group of the NaN
    bad[:, 3] = bad[:, 4] = True
    x64 = ref.act8_value(codes.cpu().numpy(), exps.cpu().numpy())
    keep = [c for c in range(d_out) if c not in (3, 4, 6)]
    fine = [r for r in range(d_in) if not 32 <= r < 64]
    assert np.isfinite(got[np.ix_(fine, keep)]).all()
    assert not np.isfinite(got[32:64]).any()
    live = np.abs(x64[7]) > 0
    assert not np.isfinite(got[:, 3][live]).any() and np.isnan(got[fine, 4]).all()
    want = x64.T @ np.where(np.isfinite(f64(dy)), f64(dy), 0.0)
    for c in (keep, [7]):
        assert rel(got[np.ix_(fine, c)], want[np.ix_(fine, c)]) <= TOL_F32
    assert got[0, 6] == float(torch.finfo(dtype).max)


# ---------------------------------------------------------- streams, graphs, memory
def all_calls(g, B=2, T=300, d=128, V=500):
    """One call of every entry point on shared inputs, as functions that return tensors."""
    ids = torch.randint(0, V, (B, T), generator=g).cuda()
    table = normal(g, V, d, dtype=BF16)
    x, dg, ig, dh = (normal(g, B, T, d, dtype=BF16) for _ in range(4))
    rate, st = torch.full((d,), 0.05, device="cuda"), normal(g, B, d)
    _, _, saved = seq.gatedrec_forward(x, dg, ig, rate, state=st, save=True)
    codes, exps = seq.act8_store(x)
    step = [t[:, :1].contiguous() for t in (x, dg, ig)]
    return {
        "embed": lambda **k: [seq.embed_forward(ids, table, 2.0, **k)],
        "embed grad": lambda **k: [seq.embed_backward(dh, ids, V, **k)],
        "recurrence": lambda **k: list(seq.gatedrec_forward(x, dg, ig, rate, state=st, save=True, **k)),
        "one token": lambda **k: list(seq.gatedrec_forward(*step, rate, state=st, **k)[:2]),
        "gradients": lambda **k: list(seq.gatedrec_backward(x, dg, ig, rate, dh, saved, **k).values()),
        "store": lambda **k: list(seq.act8_store(x, **k)),
        "load": lambda **k: [seq.act8_load(codes, exps, **k)],
        "weight grad": lambda **k: [seq.act8_weight_grad(codes, exps, dh, **k)],
    }


def test_every_call_on_another_stream():
    calls = all_calls(gen(21))
    want = {n: c() for n, c in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for n, c in calls.items():
        for s in (side, side.cuda_stream):
            got = c(stream=s)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n
    with torch.cuda.stream(side):
        for n, c in calls.items():
            got = c()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n


def test_calls_side_by_side():
    """The same operators on two streams at once, each with workspaces of its own."""
    a, b = all_calls(gen(22)), all_calls(gen(23), B=3, T=700, d=64)
    want = [{n: c() for n, c in calls.items()} for calls in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [{}, {}]
    for n in a:
        for i, calls in enumerate((a, b)):
            got[i][n] = calls[n](stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for n in a:
            assert all(torch.equal(x, y) for x, y in zip(got[i][n], want[i][n])), n


def test_every_call_in_a_graph():
    """Captured once, replayed with other inputs in between, against the eager results."""
    g = gen(24)
    B, T, d, V = 2, 300, 128, 500
    ids = torch.randint(0, V, (B, T), generator=g).cuda()
    x, dg, ig, dh = (normal(g, B, T, d, dtype=BF16) for _ in range(4))
    table, rate, st = normal(g, V, d, dtype=BF16), torch.full((d,), 0.05).cuda(), normal(g, B, d)

    def run():
        e = seq.embed_forward(ids, table, 2.0)
        h, s, saved = seq.gatedrec_forward(e, dg, ig, rate, state=st, save=True)
        codes, exps = seq.act8_store(h)
        w = seq.act8_weight_grad(codes, exps, dh)
        gr = seq.gatedrec_backward(e, dg, ig, rate, dh, saved)
        t = seq.embed_backward(gr["x"], ids, V, 2.0)
        one, s1, _ = seq.gatedrec_forward(e[:, :1], dg[:, :1], ig[:, :1], rate, state=s)
        return [e, h, s, codes, exps, seq.act8_load(codes, exps), w, *gr.values(), t, one, s1]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(4):
        ids.copy_(torch.randint(0, V, (B, T), generator=g))
        for t in (dg, ig, dh, table, st):
            t.copy_(normal(g, *t.shape, dtype=t.dtype))
        want = [t.clone() for t in run()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_workspaces_that_held_something_else():
    """A workspace's old contents mean nothing: zeros, ones, what another call left."""
    g = gen(25)
    B, T, d, V = 2, 900, 64, 300
    x, dg, ig, dh = (normal(g, B, T, d, dtype=BF16) for _ in range(4))
    ids, rate = torch.randint(0, V, (B, T), generator=g).cuda(), torch.full((d,), 0.02).cuda()
    h, s, saved = seq.gatedrec_forward(x, dg, ig, rate, save=True)
    back = seq.gatedrec_backward(x, dg, ig, rate, dh, saved)
    eg = seq.embed_backward(dh, ids, V)
    codes, exps = seq.act8_store(x)
    wg = seq.act8_weight_grad(codes, exps, dh)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127, None):
        for _ in range(2):
            if fill is not None:
                ws.fill_(fill)
            h2, s2, saved2 = seq.gatedrec_forward(x, dg, ig, rate, save=True, ws=ws)
            assert torch.equal(h2, h) and torch.equal(s2, s) and torch.equal(saved2, saved)
            if fill is not None:
                ws.fill_(fill)
            b2 = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, ws=ws)
            assert all(torch.equal(b2[n], back[n]) for n in back)
            if fill is not None:
                ws.fill_(fill)
            assert torch.equal(seq.embed_backward(dh, ids, V, ws=ws), eg)
            if fill is not None:
                ws.fill_(fill)
            assert torch.equal(seq.act8_weight_grad(codes, exps, dh, ws=ws), wg)


def test_rows_behind_the_last_are_left_alone():
    """Every output sits in front of memory that keeps its values."""
    g = gen(26)
    B, T, d, V, m = 1, 77, 72, 33, 40
    x, dg, ig, dh = (normal(g, B, T, d, dtype=BF16) for _ in range(4))
    ids, rate = torch.randint(0, V, (T,), generator=g).cuda(), torch.full((d,), 0.02).cuda()

    def room(n, dtype):
        return torch.full((n + 64,), 9, dtype=dtype, device="cuda")

    def rest(t, n):
        return (t[n:] == 9).all()

    e = seq.make_embed_desc(T, V, d, BF16)
    table, out, grad = normal(g, V, d, dtype=BF16), room(T * d, BF16), room(V * d, F32)
    seq.ttt_embed_forward(e, ids, table, out)
    e = seq.make_embed_desc(T, V, d, BF16, F32)
    ws = room(seq.ttt_embed_backward_workspace_size(e), torch.uint8)
    seq.ttt_embed_backward(e, ids, dh, grad, ws, ws.numel() - 64)
    assert rest(out, T * d) and rest(grad, V * d) and rest(ws, ws.numel() - 64)
    r = seq.make_gatedrec_desc(B, T, d, BF16)
    h, s, saved = room(T * d, BF16), room(d, F32), room(d, F32)
    ws = room(seq.ttt_gatedrec_workspace_size(r), torch.uint8)
    seq.ttt_gatedrec_forward(r, x, dg, ig, rate, None, None, s, h, saved, ws, ws.numel() - 64)
    assert rest(h, T * d) and rest(s, d) and rest(saved, d) and rest(ws, ws.numel() - 64)
    o = [room(T * d, BF16) for _ in range(3)] + [room(d, F32) for _ in range(2)]
    ws = room(seq.ttt_gatedrec_backward_workspace_size(r), torch.uint8)
    seq.ttt_gatedrec_backward(r, x, dg, ig, rate, None, saved, dh, None, *o, ws, ws.numel() - 64)
    assert all(rest(t, T * d) for t in o[:3]) and all(rest(t, d) for t in o[3:])
    assert rest(ws, ws.numel() - 64)
    a = seq.make_act8_desc(T, d, BF16)
    codes, exps, y = room(T * d, torch.int8), room(T * 3, torch.uint8), room(T * d, BF16)
    seq.ttt_act8_store(a, x, codes, exps)
    seq.ttt_act8_load(a, codes, exps, y)
    assert rest(codes, T * d) and rest(exps, T * 3) and rest(y, T * d)
    w = seq.make_act8_wgrad_desc(T, d, m, BF16)
    dy, grad = normal(g, T, m, dtype=BF16), room(d * m, F32)
    ws = room(seq.ttt_act8_weight_grad_workspace_size(w), torch.uint8)
    seq.ttt_act8_weight_grad(w, codes, exps, dy, grad, ws, ws.numel() - 64)
    assert rest(grad, d * m) and rest(ws, ws.numel() - 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [6, 400])
def test_inputs_keep_their_bits(N, dtype):
    """What a call only reads is the same to the bit behind it, infinities and NaN included."""
    g = gen(27)
    d, V, m = 72, 50, 40
    x, dg, ig, dh, dy = (normal(g, 1, N, n, dtype=dtype) for n in (d, d, d, d, m))
    rate, st, ds = torch.full((d,), 0.05, device="cuda"), normal(g, 1, d), normal(g, 1, d)
    ids, lengths = some_ids(g, N, V, torch.int64)[None].cuda(), torch.tensor([N - 1]).int().cuda()
    table = normal(g, V, d, dtype=dtype)
    rate[0], rate[1], rate[2] = -0.0, 1e30, -1.0
    for i, t in enumerate((x, dg, ig, dh, dy, table[None], st[None], ds[None])):
        t[0, -1, 3 + i], t[0, 0, 4 + i], t[0, 0, 5 + i] = float("inf"), -float("inf"), float("nan")
    codes, exps = seq.act8_store(x)
    inputs = [x, dg, ig, dh, dy, rate, st, ds, ids, lengths, table, codes, exps]
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    keep = [t.clone() for t in inputs]

    def check(name):
        for t, k in zip(inputs, keep):
            assert torch.equal(bits(t), bits(k)), name

    seq.embed_forward(ids, table, 2.0)
    check("embed_forward")
    seq.embed_backward(dh, ids, V, 2.0)
    seq.embed_backward(dh, ids, V, grad=normal(g, V, d))
    check("embed_backward")
    for ln in (None, lengths):
        _, _, saved = seq.gatedrec_forward(x, dg, ig, rate, state=st, lengths=ln, save=True)
        check("gatedrec_forward")
        old = saved.clone()
        seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=ds, lengths=ln)
        check("gatedrec_backward")
        assert torch.equal(bits(saved), bits(old))
    seq.act8_store(x)
    check("act8_store")
    seq.act8_load(codes, exps, dtype)
    check("act8_load")
    seq.act8_weight_grad(codes, exps, dy)
    seq.act8_weight_grad(codes, exps, dy, grad=normal(g, d, m))
    check("act8_weight_grad")


# ---------------------------------------------------------- offsets beyond 32 bits
def test_embed_tables_beyond_32_bits():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    V, d = 1_200_007, 2048  # 2.46e9 values, 9.8 GB in fp32
    table = torch.empty(V, d, dtype=BF16, device="cuda").normal_(generator=g)
    ids = torch.randint(0, V, (3000,), generator=g, device="cuda")
    ids[:40] = torch.arange(V - 40, V, device="cuda")
    ids[40:80] = torch.arange(40, device="cuda")
    assert torch.equal(seq.embed_forward(ids, table), table[ids])
    dout = torch.randn(3000, d, generator=g, device="cuda")
    del table
    got = seq.embed_backward(dout, ids, V, 2.0)
    rows, inverse = torch.unique(ids, return_inverse=True)
    want = torch.zeros(len(rows), d, dtype=torch.float64, device="cuda")
    want.index_add_(0, inverse, dout.double(), alpha=2.0)
    assert float((got[rows].double() - want).norm() / want.norm()) <= TOL_F32
    got[rows] = 0
    assert not got.any()
    keep = torch.ones(V, d, device="cuda")
    seq.embed_backward(dout, ids, V, 2.0, grad=keep)
    assert float((keep[rows].double() - 1 - want).norm() / want.norm()) <= TOL_F32
    keep[rows] = 1
    assert (keep == 1).all()


@pytest.mark.parametrize("N,V", [(1000, (1 << 30) + 12345), (60, (1 << 26) + 12345)])
def test_embed_backward_over_a_thousand_million_rows(N, V):
    """Every row of a gradient that takes more waves for its zeros than one launch has."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    d = 8
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    ids[:3] = torch.tensor([0, V - 1, V - 1], device="cuda")
    dout = torch.randn(N, d, generator=g, device="cuda").to(BF16)
    grad = torch.ones(V, d, dtype=BF16, device="cuda")
    desc = seq.make_embed_desc(N, V, d, BF16, BF16)
    need = seq.ttt_embed_backward_workspace_size(desc)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    seq.ttt_embed_backward(desc, ids, dout, grad, ws)
    rows, inverse = torch.unique(ids, return_inverse=True)
    want = torch.zeros(len(rows), d, dtype=torch.float64, device="cuda")
    want.index_add_(0, inverse, dout.double())
    # one rounding of a sum of one to three values of bf16, all but exact in fp32
    assert torch.equal(grad[rows], want.float().to(BF16))
    grad[rows] = 0
    assert not any(bool(part.any()) for part in grad.split(1 << 27))


def test_gatedrec_sequences_beyond_32_bits():
    """The last tokens of a call of 2^31 values and more are those of a call of their own from
    the state in front of them."""
    T, d = (1 << 20) + 300, 2056
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    new = lambda: torch.empty(1, T, d, dtype=BF16, device="cuda").normal_(generator=g)  # noqa: E731
    x, dg, ig, dh = new(), new(), new(), new()
    rate = torch.rand(d, generator=g, device="cuda") * 0.2 + 1e-3
    h, S, saved = seq.gatedrec_forward(x, dg, ig, rate, save=True)
    j = T // 128 - 3
    a = 128 * j
    last = [t[:, a:].contiguous() for t in (x, dg, ig, dh)]
    h2, S2, saved2 = seq.gatedrec_forward(*last[:3], rate, state=saved[:, j].contiguous(), save=True)
    # the state behind a tile comes by the products of its place in the call: each of the two is
    # off by TOL_F32 at most, and a bf16 result beside a tie by one step, 2^-8, more
    assert rel(f64(saved2), f64(saved[:, j:])) <= 2 * TOL_F32 and rel(f64(S2), f64(S)) <= 2 * TOL_F32
    assert rel(f64(h2), f64(h[:, a:])) <= TOL[BF16]
    ds = torch.randn(1, d, generator=g, device="cuda")
    got = seq.gatedrec_backward(x, dg, ig, rate, dh, saved, dstate_out=ds)
    want = seq.gatedrec_backward(*last[:3], rate, last[3], saved2, dstate_out=ds)
    for n in ("x", "decay_gate", "input_gate"):
        assert rel(f64(got[n][:, a:]), f64(want[n])) <= TOL[BF16], n


def test_act8_beyond_32_bits():
    rows, d = 1_100_003, 2048  # 2.25e9 values
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty(rows, d, dtype=BF16, device="cuda").normal_(generator=g)
    codes, exps = seq.act8_store(x)
    c2, e2 = seq.act8_store(x[-300:].contiguous())
    assert torch.equal(codes[-300:], c2) and torch.equal(exps[-300:], e2)
    assert torch.equal(seq.act8_load(codes, exps)[-300:], seq.act8_load(c2, e2))
    dy = torch.randn(rows, 40, generator=g, device="cuda").to(BF16)
    got = seq.act8_weight_grad(codes, exps, dy)
    want = torch.zeros(d, 40, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 100000):
        part = slice(a, a + 100000)
        want += seq.act8_load(codes[part], exps[part], F32).double().t().contiguous() @ dy[part].double()
    # sums of 1.1 million products: the slices' partial sums keep the chains short, as before
    assert float((got.double() - want).norm() / want.norm()) <= 4 * TOL_F32
