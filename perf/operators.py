"""Timed cases of the block operators: the fused residual addition and
root-mean-square norm, and linear attention with a decay for each head.

Every case is one pass through one operator, as a block around the TTT-MLP layer
calls it.  With `own` false, run() computes the operator in its plain form
(elementary torch operations in 32 bits); with `own` true it calls this
repository's kernels.  exact() gives the same outputs from the definition in 64
bits.  Sizes follow the layer's own workloads: d_model 2560 (20 heads of 128) and
1024 (16 heads of 64), 32768 and 131072 tokens, 16 sessions of 8192 tokens, 64
decoding sessions, and a tiny fp32 shape.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
EPS = 1e-6
PLAIN_CHUNK = 128  # tokens per chunk of the plain form of linear attention


# ------------------------------------------------------------------- the cases
def _attn(name, batch, seq, heads, kv_heads, dk, dv, dtype="bf16", ragged=False, state=False,
          fused=False, op="linattn"):
    return {"name": name, "op": op, "batch": batch, "seq": seq, "heads": heads,
            "kv_heads": kv_heads, "dk": dk, "dv": dv, "dtype": dtype, "ragged": ragged,
            "state": state, "fused": fused}


def _norm(name, rows, d, dtype="bf16", res="bf16", out="same", group=0, residual=True,
          op="addnorm"):
    return {"name": name, "op": op, "rows": rows, "d": d, "dtype": dtype, "res": res, "out": out,
            "group": group, "residual": residual}


def listed():
    return [
        # a 128K-token prompt of one session, q, k and v slices of one projection's output
        _attn("prompt_128k", 1, 131072, 20, 20, 128, 128, fused=True),
        # 16 sessions' prompts of up to 8K tokens in one padded batch
        _attn("prompt_16x8k_ragged", 16, 8192, 20, 20, 128, 128, ragged=True, state=True),
        # a prompt of a few hundred tokens with shared key and value heads, odd length
        _attn("prompt_777_shared", 2, 777, 16, 4, 64, 64, state=True),
        # the tiny fp32 shape
        _attn("prompt_fp32_1k", 1, 1024, 4, 4, 64, 64, dtype="fp32"),
        # one session's next token; 64 sessions' next tokens: the state is read and written
        _attn("decode_1", 1, 1, 20, 20, 128, 128, state=True),
        _attn("decode_64", 64, 1, 20, 20, 128, 128, state=True),
        # the training step's gradients at 32K tokens; and with shared heads, an odd length
        _attn("backward_32k", 1, 32768, 20, 20, 128, 128, op="linattn_bwd"),
        _attn("backward_4x1999_shared", 4, 1999, 16, 4, 64, 64, state=True, op="linattn_bwd"),
        # the norm in front of the layer at 128K tokens, and for one decoded token
        _norm("norm_128k", 131072, 2560),
        _norm("norm_decode", 1, 2560),
        # the norm in front of 8-bit projections: the residual stream in fp32, a scale per 128
        _norm("norm_fp8_32k", 32768, 2560, res="fp32", out="fp8", group=128),
        # the norm's gradients at 32K tokens
        _norm("norm_backward_32k", 32768, 2560, op="addnorm_bwd"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["prompt", "prompt", "decode", "backward", "norm", "norm_fp8", "norm_bwd"])
    if kind in ("prompt", "backward", "decode"):
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 96), (32, 64),
                             (80, 72)])
        kv = rng.choice([1, 2, 4, 5, 8, 10])
        heads = kv * rng.choice([1, 1, 1, 2, 4])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        if kind == "decode":
            batch, seq = _log_int(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 5])
            batch = max(1, min(batch, 1280 // heads))
        else:
            # tokens x heads stay below those of the largest listed case of the kind
            most = 131072 * 20 if kind == "prompt" else 32768 * 20
            most //= 16 if dtype == "fp32" else 2
            batch = _log_int(rng, 1, 16)
            seq = _log_int(rng, 17, max(18, min(131072, most // (batch * heads))))
        return _attn("", batch, seq, heads, kv, dk, dv, dtype,
                     ragged=kind == "prompt" and rng.random() < 0.4,
                     state=kind == "decode" or rng.random() < 0.5,
                     fused=kind == "prompt" and rng.random() < 0.4,
                     op="linattn_bwd" if kind == "backward" else "linattn")
    d = rng.choice([64, 128, 200, 1024, 1536, 2560, 4096, 5120, 8192, 9728])
    rows = _log_int(rng, 1, min(131072, 131072 * 1280 // d))
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    res = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
    if kind == "norm_fp8":
        return _norm("", rows, d, dtype, res, "fp8",
                     128 if d % 128 == 0 and rng.random() < 0.5 else 0, rng.random() < 0.8)
    if kind == "norm_bwd":
        return _norm("", rows, d, dtype, res, residual=rng.random() < 0.8, op="addnorm_bwd")
    return _norm("", rows, d, dtype, res, residual=rng.random() < 0.8)


# ------------------------------------------------------------------ the inputs
def _inputs(case, seed):
    """The inputs of a case from its seed, a dict of device tensors."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    if case["op"].startswith("addnorm"):
        rows, d = case["rows"], case["d"]
        rdt = DTYPES[case["res"]]
        s = {"weight": (1.0 + 0.1 * torch.randn(d, generator=g, device=dev)).to(dt)}
        if case["op"] == "addnorm":
            s["x"] = normal(rows, d, dtype=dt)
            # a residual stream grows over the blocks before
            s["res"] = normal(rows, d, dtype=rdt, std=3.0) if case["residual"] else None
        else:
            s["r"] = normal(rows, d, dtype=rdt, std=3.0)
            s["dy"] = normal(rows, d, dtype=dt)
            # the gradient that reaches the sum from the blocks after
            s["dr"] = normal(rows, d, dtype=rdt) if case["residual"] else None
        return s

    B, T, H, G = case["batch"], case["seq"], case["heads"], case["kv_heads"]
    dk, dv = case["dk"], case["dv"]
    silu = torch.nn.functional.silu
    if case["fused"]:  # slices of one projection's rows
        w = H * dk + G * dk + G * dv
        x = torch.empty(B, T, w, device=dev, dtype=dt)
        x.copy_(normal(B, T, w, dtype=dt))
        qk = x[..., :(H + G) * dk]
        qk.copy_(silu(qk.float()).to(dt))
        q = x[..., :H * dk].unflatten(-1, (H, dk))
        k = x[..., H * dk:(H + G) * dk].unflatten(-1, (G, dk))
        v = x[..., (H + G) * dk:].unflatten(-1, (G, dv))
    else:
        q = silu(normal(B, T, H, dk)).to(dt)
        k = silu(normal(B, T, G, dk)).to(dt)
        v = normal(B, T, G, dv, dtype=dt)
    # memories from about one token to some thousand tokens, as fixed slopes give them
    i = torch.arange(H, device=dev, dtype=torch.float32)
    s = {"q": q, "k": k, "v": v, "log_decay": -torch.exp2(-1.0 - 10.0 * (i + 0.5) / H),
         "scale": dk ** -0.5, "lengths": None, "state": None}
    if case["ragged"]:
        s["lengths"] = torch.randint(T // 2, T + 1, (B,), generator=g, device=dev,
                                     dtype=torch.int32)
    if case["state"]:
        s["state"] = normal(B, H, dk, dv, std=2.0)
    if case["op"] == "linattn_bwd":
        s["dO"] = normal(B, T, H, dv, dtype=dt)
        s["dstate"] = normal(B, H, dk, dv, std=0.1) if case["state"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# -------------------------------------------------------------- the plain forms
def _spread(x, H):
    """[B][T][G][D] -> [B][H][T][D] fp32, each kv head repeated for its query heads."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(H // x.shape[1], dim=1) if x.shape[1] != H else x


def _chunks(x, n):
    """[B][H][T][D] -> [B][H][n][C][D], zeros behind T."""
    B, H, T, D = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, n * PLAIN_CHUNK - T))
    return x.reshape(B, H, n, PLAIN_CHUNK, D)


def _power(lg, n):
    """decay^n, 1 where n is 0, 0 where n is negative; lg broadcast in front of n."""
    return torch.where(n > 0, torch.exp(lg * n.clamp(min=0)), (n == 0).to(lg.dtype))


def _scan(q, k, v, lg, state, late):
    """o_t = sum_{s <= t} decay^(t-s) (q_t . k_s) v_s + decay^(t+late) q_t state over tokens
    [B][H][T][D], in chunks side by side; and the state behind the last token."""
    B, H, T, dk = q.shape
    C, dev = PLAIN_CHUNK, q.device
    n = -(-T // C)
    q, k, v = _chunks(q, n), _chunks(k, n), _chunks(v, n)
    lg = lg.view(1, H, 1, 1)
    i = torch.arange(C, device=dev)
    inside = _power(lg, i[:, None] - i[None, :]).unsqueeze(2)            # [1][H][1][C][C]
    o = ((q @ k.transpose(-1, -2)) * inside) @ v
    to_end = _power(lg, (C - 1 + (1 - late) - i)[None, :]).view(1, H, 1, C, 1)
    inc = (k * to_end).transpose(-1, -2) @ v                            # [B][H][n][dk][dv]
    j = torch.arange(n, device=dev)
    before = _power(lg, C * (j[:, None] - 1 - j[None, :])).view(1, H, n, n)
    S = (before @ inc.reshape(B, H, n, -1)).reshape(inc.shape)
    if state is not None:
        S = S + _power(lg, C * j[:, None]).view(1, H, n, 1, 1) * state.unsqueeze(2)
    o = o + _power(lg, (i + late)[:, None]).view(1, H, 1, C, 1) * (q @ S)
    o = o.reshape(B, H, n * C, -1)[:, :, :T]
    # behind token T - 1: the last chunk holds m of its C tokens
    m = T - (n - 1) * C
    last = _power(lg, (m - 1 + (1 - late) - i)[None, :]).view(1, H, C, 1)
    end = (k[:, :, -1] * last).transpose(-1, -2) @ v[:, :, -1]
    return o, end + _power(lg, torch.tensor([[m]], device=dev)).view(1, H, 1, 1) * S[:, :, -1]


def _plain_linattn(s):
    q, k, v, lg, st, ln = s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["lengths"]
    H, T = q.shape[2], q.shape[1]
    qf, kf, vf = _spread(q, H), _spread(k, H), _spread(v, H)
    if T == 1 and ln is None:
        new = kf.transpose(-1, -2) @ vf
        if st is not None:
            new = new + torch.exp(lg).view(1, H, 1, 1) * st
        o = qf @ new
    elif ln is None:
        o, new = _scan(qf, kf, vf, lg, st, 1)
    else:
        # sequences moved to the end of their rows: a zero token only decays the state, so the
        # state given enters behind those in front
        t = torch.arange(T, device=q.device)
        pad = (T - ln.long()).view(-1, 1)
        at = t[None, :] - pad                                            # token, < 0: none
        pick = lambda x: torch.gather(x, 2, at.clamp(min=0)[:, None, :, None].expand_as(x))  # noqa: E731
        live = (at >= 0)[:, None, :, None]
        zero = torch.zeros((), device=q.device)
        qs, ks, vs = (torch.where(live, pick(x), zero) for x in (qf, kf, vf))
        o, new = _scan(qs, ks, vs, lg, None, 1)
        if st is not None:
            since = _power(lg.view(1, H, 1), (at + 1).clamp(min=0)[:, None, :]).unsqueeze(-1)
            o = o + torch.where(live, since * (qs @ st), zero)
            new = new + _power(lg.view(1, H), ln.view(-1, 1)).view(-1, H, 1, 1) * st
        back = (t[None, :] + pad).clamp(max=T - 1)
        o = torch.gather(o, 2, back[:, None, :, None].expand_as(o))
        o = torch.where((t[None, :] < ln.view(-1, 1))[:, None, :, None], o, zero)
    o = (o * s["scale"]).transpose(1, 2).to(q.dtype).contiguous()
    if st is not None:
        st.copy_(new)
        new = st
    return {"o": o, "state": new}


def _plain_linattn_bwd(s):
    q, k, v, lg, st, sc = s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["scale"]
    H, G = q.shape[2], k.shape[2]
    qf, kf, vf, df = _spread(q, H), _spread(k, H), _spread(v, H), _spread(s["dO"], H) * sc
    back = lambda x: x.flip(2)  # noqa: E731
    ds = s["dstate"]
    # dq is the operator itself with (dO, v, k) for (q, k, v); dk and dv run from the last token
    dq, _ = _scan(df, vf, kf, lg, None if st is None else st.transpose(-1, -2), 1)
    dk, _ = _scan(back(vf), back(df), back(qf), lg, None if ds is None else ds.transpose(-1, -2), 0)
    dv, dst = _scan(back(kf), back(qf), back(df), lg, ds, 0)

    def out(x, heads, like):
        x = x.reshape(x.shape[0], heads, H // heads, x.shape[2], x.shape[3]).sum(2)
        return x.transpose(1, 2).to(like.dtype).contiguous()

    return {"dq": out(dq, H, q), "dk": out(back(dk), G, k), "dv": out(back(dv), G, v),
            "dstate": dst if st is not None else None}


def _plain_addnorm(s):
    c = s["case"]
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {"r": None if s["res"] is None else r.to(s["res"].dtype)}
    if c["out"] == "same":
        return out | {"y": y.to(s["x"].dtype)}
    g = c["group"] or c["d"]
    y = y.unflatten(-1, (c["d"] // g, g))
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
    return out | {"y": (y / scale).flatten(-2).to(FP8), "scale": scale.squeeze(-1)}


def _plain_addnorm_bwd(s):
    r, dy, w = s["r"].float(), s["dy"].float(), s["weight"].float()
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    n = r * rstd
    dw = (dy * n).sum(0)
    g = dy * w
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    out = {"dr": dx.to(s["r"].dtype), "dweight": dw}
    if s["dy"].dtype != s["r"].dtype:
        out["dx"] = dx.to(s["dy"].dtype)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        from chunk_wise_weight_chunked_amd import block
        if op == "linattn":
            st = state["state"]
            o, st = block.linattn_forward(state["q"], state["k"], state["v"], state["log_decay"],
                                          scale=state["scale"], state=st, state_out=st,
                                          lengths=state["lengths"])
            return {"o": o, "state": st}
        if op == "linattn_bwd":
            g = block.linattn_backward(state["q"], state["k"], state["v"], state["log_decay"],
                                       state["dO"], scale=state["scale"], state=state["state"],
                                       dstate_out=state["dstate"])
            return {"dq": g["q"], "dk": g["k"], "dv": g["v"], "dstate": g["state"]}
        if op == "addnorm":
            c = state["case"]
            y, r, scale = block.add_rmsnorm(state["x"], state["res"], state["weight"], EPS,
                                            out_dtype=FP8 if c["out"] == "fp8" else None,
                                            scale_group=c["group"])
            return {"r": r, "y": y} | ({} if scale is None else {"scale": scale})
        dr, dx, dw = block.add_rmsnorm_backward(state["dy"], state["r"], state["weight"], EPS,
                                                dr=state["dr"])
        return {"dr": dr, "dweight": dw} | ({} if dx is dr else {"dx": dx})
    return {"linattn": _plain_linattn, "linattn_bwd": _plain_linattn_bwd,
            "addnorm": _plain_addnorm, "addnorm_bwd": _plain_addnorm_bwd}[op](state)


# ------------------------------------------------------------------------ work
def work(case):
    es = {"bf16": 2, "fp32": 4}
    e = es[case["dtype"]]
    if case["op"].startswith("addnorm"):
        n, er = case["rows"] * case["d"], es[case["res"]]
        if case["op"] == "addnorm":
            eo = 1 if case["out"] == "fp8" else e
            b = n * (e + eo + (2 * er if case["residual"] else 0))
            if case["out"] == "fp8":
                b += 4 * n // (case["group"] or case["d"])
            return {"bytes": b + case["d"] * e, "flops": 5 * n}
        b = n * (e + er + er + (er if case["residual"] else 0) + (e if e != er else 0))
        return {"bytes": b + case["d"] * (e + 4), "flops": 12 * n}
    B, T, H, G = case["batch"], case["seq"], case["heads"], case["kv_heads"]
    dk, dv = case["dk"], case["dv"]
    live = 0.75 if case["ragged"] else 1.0
    st = 4 * B * H * dk * dv
    io = B * T * (H * (dk + dv) + G * (dk + dv)) * e
    if case["op"] == "linattn":
        return {"bytes": io * live + st * (2 if case["state"] else 1),
                "flops": live * B * T * H * 4 * dk * dv}
    # q, k, v and dO read, dq, dk and dv written; four state products of the recurrence more
    return {"bytes": 2 * io - B * T * H * dv * e + (3 * st if case["state"] else 0),
            "flops": B * T * H * 10 * dk * dv}


# ------------------------------------------------------- the definition in 64 bits
def _recur64(q, k, v, lg, st, ln):
    """The recurrence S_t = decay S_{t-1} + k_t v_t, o_t = q_t S_t in blocks of 64 tokens one
    after the other, [B][T][H][D] in 64 bits; tokens at ln or behind it do nothing."""
    B, T, H, _ = q.shape
    S, outs = st, []
    lg = lg.view(1, 1, H)
    t = torch.arange(T, device=q.device)
    live = (t[None, :] < ln[:, None])
    step = live.double()[..., None] * lg.clamp(min=-1e4)                 # [B][T][H]
    for a in range(0, T, 64):
        m = live[:, a:a + 64, None, None]
        qb, kb, vb = (torch.where(m, x[:, a:a + 64].double(), 0.0).transpose(1, 2)
                      for x in (q, k, v))
        c = step[:, a:a + 64].cumsum(1).transpose(1, 2)                  # [B][H][b]
        n = c.shape[-1]
        low = torch.ones(n, n, device=q.device, dtype=torch.bool).tril()
        w = torch.where(low, c[..., :, None] - c[..., None, :], -math.inf).exp()
        o = ((qb @ kb.transpose(-1, -2)) * w) @ vb + c.exp()[..., None] * (qb @ S)
        outs.append(torch.where(m.transpose(1, 2), o, 0.0).transpose(1, 2))
        to_end = (c[..., -1:] - c).exp()[..., None]
        S = c[..., -1].exp()[..., None, None] * S + (kb * to_end).transpose(-1, -2) @ vb
    return torch.cat(outs, 1), S


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "addnorm":
        r = s["x"].double()
        if s["res"] is not None:
            r = r + s["res"].double()
        y = r / (r.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * s["weight"].double()
        out = {"r": None if s["res"] is None else r}
        if case["out"] == "same":
            return out | {"y": y}
        g = case["group"] or case["d"]
        y = y.reshape(case["rows"], -1, g)
        scale = y.abs().max(-1, keepdim=True).values / FP8_MAX
        return out | {"y": (y / scale).reshape(case["rows"], -1), "scale": scale[..., 0]}
    if case["op"] == "addnorm_bwd":
        r = s["r"].double().requires_grad_(True)
        w = s["weight"].double().requires_grad_(True)
        y = r / (r.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * w
        dr, dw = torch.autograd.grad(y, (r, w), s["dy"].double())
        if s["dr"] is not None:
            dr = dr + s["dr"].double()
        return {"dr": dr, "dweight": dw} | ({"dx": dr} if case["dtype"] != case["res"] else {})

    B, T, H = case["batch"], case["seq"], case["heads"]
    rep = H // case["kv_heads"]
    q, k, v = s["q"], s["k"], s["v"]
    st = s["state"].double() if s["state"] is not None else torch.zeros(
        B, H, case["dk"], case["dv"], dtype=torch.float64, device=q.device)
    ln = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    lg = s["log_decay"].double()
    shared = lambda x: x.repeat_interleave(rep, dim=2)  # noqa: E731
    if case["op"] == "linattn":
        o, end = _recur64(q, shared(k), shared(v), lg, st, ln)
        return {"o": o * s["scale"], "state": end}
    leaf = [x.double().requires_grad_(True) for x in (q, k, v, st)]
    o, end = _recur64(leaf[0], shared(leaf[1]), shared(leaf[2]), lg, leaf[3], ln)
    seeds = [s["dO"].double() * s["scale"],
             s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(end)]
    dq, dk, dv, dst = torch.autograd.grad((o, end), leaf, seeds)
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": dst if s["state"] is not None else None}
