"""Timed cases of the sequence operators: the embedding lookup and its gradient, the gated
linear recurrence with its gradients, and activations kept in 8 bits for the backward pass.

Every case is one pass through one operator (a training step of the recurrence: forward and
gradients), as a stack of blocks around the TTT-MLP layer calls it.  With `own` false, run()
computes the operator in its plain form (elementary torch operations in 32 bits); with `own` true
it calls this repository's kernels.  exact() gives the same outputs from the definition in 64 bits.
Sizes follow the layer's own workloads: d_model 2560 and 1024, 32768 and 131072 tokens, 16 sessions
of 8192 tokens, 64 decoding sessions; vocabularies are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GROUP = 32  # values of a row that share a scale in 8 bits


# ------------------------------------------------------------------- the cases
def _embed(name, op, tokens, vocab, d, dtype="bf16", out="same", add=False):
    return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "d": d, "dtype": dtype,
            "out": out, "add": add}


def _recur(name, op, batch, seq, d, dtype="bf16", ragged=False, state=False, fused=False):
    return {"name": name, "op": op, "batch": batch, "seq": seq, "d": d, "dtype": dtype,
            "ragged": ragged, "state": state, "fused": fused}


def _act8(name, op, rows, d, d_out=0, dtype="bf16", grad="fp32", add=False):
    return {"name": name, "op": op, "rows": rows, "d": d, "d_out": d_out, "dtype": dtype,
            "grad": grad, "add": add}


def listed():
    return [
        # the embeddings of a 128K-token prompt; of 64 sessions' next tokens, into an fp32 stream
        _embed("embed_128k", "embed", 131072, 65536, 2560),
        _embed("embed_decode_64", "embed", 64, 65536, 2560, out="fp32"),
        # the table's gradient of a 32K-token training step, whole; and added to one that is there
        # already (a table shared with the output projection), of 16 sequences of odd length
        _embed("embed_grad_32k", "embed_bwd", 32768, 50001, 2560, out="fp32"),
        _embed("embed_grad_add_16x1999", "embed_bwd", 16 * 1999, 131072, 1024, out="fp32",
               add=True),
        # a 128K-token prompt of one session, x and the gates slices of one projection's output
        _recur("recur_128k", "recur", 1, 131072, 2560, fused=True),
        # 64 sessions' next tokens: the state is read and written
        _recur("recur_decode_64", "recur", 64, 1, 2560, state=True),
        # training steps: 32K tokens; a padded batch in fp32 of odd length
        _recur("recur_train_32k", "recur_train", 1, 32768, 2560),
        _recur("recur_train_4x1999_fp32", "recur_train", 4, 1999, 1024, dtype="fp32", ragged=True,
               state=True),
        # a 32K-token activation into 8 bits, and a small one
        _act8("act8_store_32k", "act8_store", 32768, 2560),
        _act8("act8_store_777", "act8_store", 777, 1000, dtype="fp32"),
        # the gradient of the projection of q, k and v at 32K tokens; a smaller one in fp32, added
        _act8("act8_wgrad_32k", "act8_wgrad", 32768, 2560, 7680),
        _act8("act8_wgrad_1554_fp32", "act8_wgrad", 1554, 1024, 1536, dtype="fp32", add=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["embed", "embed_bwd", "recur", "recur_train", "recur_train", "decode",
                       "act8_store", "act8_wgrad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    d = rng.choice([64, 200, 1000, 1024, 1536, 2048, 2560, 4096, 5120])
    if kind == "embed":
        return _embed("", kind, _log_int(rng, 1, 131072 * 1280 // max(d, 1280)),
                      _log_int(rng, 1000, 131072), d, dtype, rng.choice(["same", "fp32"]))
    if kind == "embed_bwd":
        # the dense gradient of the largest listed case is 50001 rows of 2560
        return _embed("", kind, _log_int(rng, 1, 32768 * 1280 // max(d, 1280)),
                      _log_int(rng, 1000, min(131072, 50001 * 2560 // d)), d, dtype,
                      rng.choice(["same", "fp32", "fp32"]), rng.random() < 0.4)
    if kind == "decode":
        return _recur("", "recur", _log_int(rng, 1, 64), rng.choice([1, 1, 2, 3, 5]), d, dtype,
                      state=True)
    if kind in ("recur", "recur_train"):
        most = (131072 if kind == "recur" else 32768) * 2560 // d // (1 if dtype == "bf16" else 2)
        batch = _log_int(rng, 1, 16)
        return _recur("", kind, batch, _log_int(rng, 7, max(8, min(131072, most // batch))), d,
                      dtype, rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.4)
    if kind == "act8_store":
        return _act8("", kind, _log_int(rng, 1, 32768 * 1280 // max(d, 1280)), d, dtype=dtype)
    d_out = rng.choice([64, 328, 1024, 1536, 2560, 4096, 7680])
    most = min(32768, 32768 * 2560 * 7680 // (d * d_out)) // (1 if dtype == "bf16" else 4)
    add = rng.random() < 0.3
    return _act8("", kind, _log_int(rng, 1, most), d, d_out, dtype,
                 "fp32" if add or dtype == "fp32" else rng.choice(["fp32", "bf16"]), add)


# ------------------------------------------------------------------ the inputs
def _inputs(case, seed):
    """The inputs of a case from its seed, a dict of device tensors."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    if case["op"].startswith("embed"):
        N, V, d = case["tokens"], case["vocab"], case["d"]
        # frequencies of tokens fall like 1 / rank: the ranks spread over their logarithm, and
        # over the table's rows by a fixed permutation of the vocabulary
        u = torch.rand(N, generator=g, device=dev, dtype=torch.float64)
        rank = torch.exp(u * math.log(V)).long().clamp(1, V) - 1
        ids = (rank * 48271 + 11) % V if math.gcd(48271, V) == 1 else rank
        s = {"ids": ids, "vocab": V, "scale": math.sqrt(d),
             "out_dtype": dt if case["out"] == "same" else torch.float32}
        if case["op"] == "embed":
            return s | {"table": normal(V, d, dtype=dt, std=d ** -0.5)}
        s["dout"] = normal(N, d, dtype=dt)
        # what the output projection's gradient left in a shared table's
        s["grad"] = normal(V, d, dtype=s["out_dtype"]) if case["add"] else None
        return s
    if case["op"].startswith("act8"):
        n, d = case["rows"], case["d"]
        # activations: a few channels are much larger than the others
        x = normal(n, d) * torch.exp(0.7 * torch.randn(d, generator=g, device=dev))
        s = {"x": x.to(dt)}
        if case["op"] == "act8_wgrad":
            s["codes"], s["exps"] = _plain_store(s.pop("x"))
            s["dy"] = normal(n, case["d_out"], dtype=dt)
            s["grad_dtype"] = DTYPES[case["grad"]]
            # what earlier parts of the batch left in the gradient
            s["grad"] = normal(d, case["d_out"], std=n ** 0.5) if case["add"] else None
        return s

    B, T, d = case["batch"], case["seq"], case["d"]
    if case["fused"]:  # slices of one projection's rows, an output gate's behind them
        p = normal(B, T, 4 * d, dtype=dt)
        x, ga, gi = p[..., :d], p[..., d:2 * d], p[..., 2 * d:3 * d]
    else:
        x, ga, gi = (normal(B, T, d, dtype=dt) for _ in range(3))
    # memories from about one token to some thousand tokens
    s = {"x": x, "ga": ga, "gi": gi, "lengths": None, "state": None,
         "rate": torch.exp(torch.empty(d, device=dev).uniform_(math.log(1e-3), math.log(2.0),
                                                               generator=g))}
    if case["ragged"]:
        s["lengths"] = torch.randint(T // 2, T + 1, (B,), generator=g, device=dev,
                                     dtype=torch.int32)
    if case["state"]:
        s["state"] = normal(B, d)
    if case["op"] == "recur_train":
        s["dh"] = normal(B, T, d, dtype=dt)
        s["dstate"] = normal(B, d) if case["state"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# -------------------------------------------------------------- the plain forms
def _plain_embed(s):
    ids, V = s["ids"], s["vocab"]
    live = ((ids >= 0) & (ids < V)).unsqueeze(-1)
    rows = s["table"][ids.clamp(0, V - 1)].float() * s["scale"]
    return {"out": torch.where(live, rows, 0.0).to(s["out_dtype"])}


def _plain_embed_bwd(s):
    ids, V, d = s["ids"], s["vocab"], s["dout"].shape[-1]
    live = ((ids >= 0) & (ids < V)).unsqueeze(-1)
    rows = torch.where(live, s["dout"].float() * s["scale"], 0.0)
    ids = ids.clamp(0, V - 1)
    if s["grad"] is None:
        return {"grad": torch.zeros(V, d, device=ids.device).index_add_(0, ids, rows)
                .to(s["out_dtype"])}
    if s["out_dtype"] == torch.float32:
        return {"grad": s["grad"].index_add_(0, ids, rows)}
    return {"grad": s["grad"].copy_(s["grad"].float().index_add_(0, ids, rows))}


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t over dimension 1, from h = 0: neighbours are joined to pairs, the
    pairs' scan gives every second value, one more step the others."""
    T = u.shape[1]
    if T == 1:
        return u
    n = T // 2 * 2
    odd = _scan(a[:, 1:n:2] * a[:, 0:n:2], u[:, 1:n:2] + a[:, 1:n:2] * u[:, 0:n:2])
    h = torch.empty_like(u)
    h[:, 1::2] = odd
    h[:, :1] = u[:, :1]
    h[:, 2::2] = u[:, 2::2] + a[:, 2::2] * odd[:, :(T + 1) // 2 - 1]
    return h


def _parts(s):
    """x, r, i, z, a, b and the tokens that count, of the recurrence.  a is in 64 bits: the rounding
    of a decay near 1 would be repeated over all tokens that a channel remembers."""
    x, T = s["x"].float(), s["x"].shape[1]
    r, i = torch.sigmoid(s["ga"].float()), torch.sigmoid(s["gi"].float())
    z = -s["rate"] * r
    b = torch.sqrt(-torch.expm1(2 * z))
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(T, device=x.device)[None, :] < s["lengths"].long()[:, None])[..., None]
        z, b = torch.where(live, z, 0.0), torch.where(live, b, 0.0)
    return x, r, i, z, torch.exp(z.double()), b, live


def _plain_recur(s):
    x, r, i, z, a, b, live = _parts(s)
    u = (b * i * x).double()
    if s["state"] is not None:
        u[:, 0] += a[:, 0] * s["state"]
    h = _scan(a, u)
    state = h[:, -1].float()
    out = h if live is None else torch.where(live, h, 0.0)
    return {"h": out.to(s["x"].dtype), "state": state}, h, (x, r, i, z, a, b, live)


def _plain_recur_forward(s):
    out = _plain_recur(s)[0]
    if s["state"] is not None:
        out["state"] = s["state"].copy_(out["state"])
    return out


def _plain_recur_train(s):
    out, h, (x, r, i, z, a, b, live) = _plain_recur(s)
    first = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    dh = s["dh"].double()
    if live is not None:
        dh = torch.where(live, dh, 0.0)
    if s["dstate"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dstate"][:, None]], 1)
    after = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    lam = _scan(after, dh.flip(1)).flip(1)
    # the derivative of b = sqrt(1 - a^2) is taken as 0 where b is 0
    inv = torch.where(b > 0, 1 / b, 0.0)
    dz = lam * (a * before - i * x * a * a * inv)
    if live is not None:
        dz = torch.where(live, dz, 0.0)
    dt = s["x"].dtype
    return out | {"dx": (lam * b * i).to(dt), "dga": (dz * z * (1 - r)).to(dt),
                  "dgi": (lam * b * i * x * (1 - i)).to(dt), "drate": -(dz * r).sum((0, 1)).float(),
                  "dstate": None if s["state"] is None else (a * lam)[:, 0].float()}


def _plain_store(x):
    n, d = x.shape
    groups = -(-d // GROUP)
    g = torch.nn.functional.pad(x.float(), (0, groups * GROUP - d)).view(n, groups, GROUP)
    top = g.abs().amax(-1, keepdim=True)
    # the smallest power of two 2^e, e >= -126, that takes the largest value to at most 127:
    # top = m 2^k with m in [0.5, 1), so that top / 2^(k - 7) is in [64, 128)
    m, k = torch.frexp(top)
    e = torch.where(top > 0, (k - 7 + (m > 127 / 128)).clamp(min=-126), -126).to(torch.int32)
    codes = torch.round(g * ((127 - e) << 23).view(torch.float32))
    fine = torch.isfinite(top)
    codes = torch.where(fine, codes, 0.0).to(torch.int8).view(n, -1)[:, :d].contiguous()
    return codes, torch.where(fine, e + 127, 255).to(torch.uint8).view(n, groups)


def _plain_act8_store(s):
    codes, exps = _plain_store(s["x"])
    return {"codes": codes, "exps": exps}


def _plain_act8_wgrad(s):
    d = s["codes"].shape[1]
    scale = (s["exps"].int() << 23).view(torch.float32).repeat_interleave(GROUP, 1)[:, :d]
    grad = (s["codes"].float() * scale).t() @ s["dy"].float()
    if s["grad"] is not None:
        return {"grad": s["grad"].add_(grad)}
    return {"grad": grad.to(s["grad_dtype"])}


def run(state):
    op = state["case"]["op"]
    if own:
        from chunk_wise_weight_chunked_amd import seq
        if op == "embed":
            return {"out": seq.embed_forward(state["ids"], state["table"], state["scale"],
                                             out_dtype=state["out_dtype"])}
        if op == "embed_bwd":
            return {"grad": seq.embed_backward(state["dout"], state["ids"], state["vocab"],
                                               state["scale"], grad_dtype=state["out_dtype"],
                                               grad=state["grad"])}
        if op == "recur":
            st = state["state"]
            h, st, _ = seq.gatedrec_forward(state["x"], state["ga"], state["gi"], state["rate"],
                                            state=st, state_out=st, lengths=state["lengths"])
            return {"h": h, "state": st}
        if op == "recur_train":
            h, st, saved = seq.gatedrec_forward(state["x"], state["ga"], state["gi"],
                                                state["rate"], state=state["state"],
                                                lengths=state["lengths"], save=True)
            g = seq.gatedrec_backward(state["x"], state["ga"], state["gi"], state["rate"],
                                      state["dh"], saved, dstate_out=state["dstate"],
                                      lengths=state["lengths"])
            return {"h": h, "state": st, "dx": g["x"], "dga": g["decay_gate"],
                    "dgi": g["input_gate"], "drate": g["rate"],
                    "dstate": None if state["state"] is None else g["state"]}
        if op == "act8_store":
            codes, exps = seq.act8_store(state["x"])
            return {"codes": codes, "exps": exps}
        return {"grad": seq.act8_weight_grad(state["codes"], state["exps"], state["dy"],
                                             grad_dtype=state["grad_dtype"],
                                             grad=state["grad"])}
    return {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "recur": _plain_recur_forward,
            "recur_train": _plain_recur_train, "act8_store": _plain_act8_store,
            "act8_wgrad": _plain_act8_wgrad}[op](state)


# ------------------------------------------------------------------------ work
def work(case):
    es = {"bf16": 2, "fp32": 4}
    e = es[case["dtype"]]
    if case["op"].startswith("embed"):
        N, V, d = case["tokens"], case["vocab"], case["d"]
        eo = e if case["out"] == "same" else 4
        # rows that N draws over the logarithm of the rank reach: rank k with probability
        # log(1 + 1 / k) / log V each time
        k = torch.arange(1, V + 1, dtype=torch.float64)
        rows = float((1 - (1 - torch.log1p(1 / k) / math.log(V)) ** N).sum())
        if case["op"] == "embed":
            return {"bytes": N * (8 + d * eo) + rows * d * e, "flops": N * d}
        return {"bytes": N * (8 + d * e) + d * eo * (2 * rows if case["add"] else V),
                "flops": N * d}
    if case["op"].startswith("act8"):
        n, d, m = case["rows"], case["d"], case["d_out"]
        kept = n * d + n * -(-d // GROUP)
        if case["op"] == "act8_store":
            return {"bytes": n * d * e + kept, "flops": 3 * n * d}
        eg = es[case["grad"]]
        return {"bytes": kept + n * m * e + d * m * eg * (2 if case["add"] else 1),
                "flops": 2 * n * d * m}
    B, T, d = case["batch"], case["seq"], case["d"]
    live = 0.75 if case["ragged"] else 1.0
    n, st = B * T * d * live, 4 * B * d
    if case["op"] == "recur":
        return {"bytes": 4 * n * e + st * (2 if case["state"] else 1) + 4 * d, "flops": 30 * n}
    # forward 3 read and 1 written, gradients 4 read and 3 written
    return {"bytes": 11 * n * e + st * (4 if case["state"] else 1) + 12 * d, "flops": 100 * n}


# ------------------------------------------------------- the definition in 64 bits
def _recur64(a, u, first):
    """h_t = a_t h_{t-1} + u_t over [B][T][d] in 64 bits: parts of the sequence side by side, one
    token after the other, and then each part's start into its tokens."""
    B, T, d = u.shape
    L = max(1, math.isqrt(T))
    n = -(-T // L)
    pad = n * L - T
    a = torch.nn.functional.pad(a, (0, 0, 0, pad), value=1.0).view(B, n, L, d)
    h = torch.nn.functional.pad(u, (0, 0, 0, pad)).view(B, n, L, d).clone()
    keep = a.clone()
    for t in range(1, L):
        h[:, :, t] += a[:, :, t] * h[:, :, t - 1]
        keep[:, :, t] *= keep[:, :, t - 1]
    start = first
    for j in range(n):
        h[:, j] += keep[:, j] * start[:, None]
        start = h[:, j, -1]
    return h.view(B, n * L, d)[:, :T]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "embed":
        return {"out": s["table"].double().index_select(0, s["ids"]) * s["scale"]}
    if case["op"] == "embed_bwd":
        grad = torch.zeros(case["vocab"], case["d"], dtype=torch.float64, device=s["ids"].device)
        if s["grad"] is not None:
            grad += s["grad"].double()
        return {"grad": grad.index_add_(0, s["ids"], s["dout"].double(), alpha=s["scale"])}
    if case["op"] == "act8_store":
        x = s["x"].double()
        n, d = x.shape
        x = torch.cat([x, x.new_zeros(n, -d % GROUP)], 1).view(n, -1, GROUP)
        top = x.abs().max(-1, keepdim=True).values
        e = torch.ceil(torch.log2(top / 127)).clamp(min=-126.0)
        codes = torch.round(x / torch.exp2(e)).view(n, -1)[:, :d]
        return {"codes": codes.to(torch.int8), "exps": (e[..., 0] + 127).to(torch.uint8)}
    if case["op"] == "act8_wgrad":
        k = torch.arange(case["d"], device=s["codes"].device) // GROUP
        x = torch.ldexp(s["codes"].double(), s["exps"].int()[:, k] - 127)
        grad = x.t().contiguous() @ s["dy"].double()
        return {"grad": grad if s["grad"] is None else grad + s["grad"].double()}

    B, T, d = case["batch"], case["seq"], case["d"]
    x, r, i = s["x"].double(), s["ga"].double().sigmoid(), s["gi"].double().sigmoid()
    rate = s["rate"].double()
    dev = x.device
    ln = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=dev)
    gone = (torch.arange(T, device=dev) >= ln[:, None])[..., None]
    a = (-rate * r).exp().masked_fill_(gone, 1.0)
    b = (-(-2 * rate * r).expm1()).sqrt().masked_fill_(gone, 0.0)
    first = s["state"].double() if s["state"] is not None else torch.zeros(B, d, device=dev,
                                                                           dtype=torch.float64)
    h = _recur64(a, b * i * x, first)
    out = {"h": h.masked_fill(gone, 0.0), "state": h[:, -1]}
    if case["op"] == "recur":
        return out
    # the sum of what each h_t gives the loss, through h_t alone and through those after it
    dh = s["dh"].double().masked_fill(gone, 0.0)
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    end = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(first)
    lam = _recur64(later.flip(1), dh.flip(1), end).flip(1)
    del dh, later
    h = torch.cat([first[:, None], h[:, :-1]], 1)
    slope = torch.where(b > 0, a * a / b, 0.0)
    dz = (lam * (a * h - i * x * slope)).masked_fill_(gone, 0.0)
    return out | {"dx": lam * b * i, "dga": dz * (-rate * r) * (1 - r),
                  "dgi": lam * b * x * i * (1 - i), "drate": -(dz * r).sum((0, 1)),
                  "dstate": None if s["state"] is None else (a * lam)[:, 0]}
