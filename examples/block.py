"""A block around the TTT-MLP layer from this library's operators: a prompt, the
tokens after it, and one training step.

    python examples/block.py

    r = x + residual, y = norm(r)          add_rmsnorm
    q, k, v = y W_qkv (SiLU on q and k)    the caller's matrix product
    o = linear attention of q, k, v        linattn_forward, a state per session
    r = r + o W_o, h = norm(r)             add_rmsnorm
    out = TTT-MLP(h)                       ttt_mlp.forward_batched / Stream

Served, a session keeps two things of constant size: the attention's state and
the layer's fast weight.  Trained, every part has its gradient; the parts in
between (projections, SiLU) are elementary torch.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from chunk_wise_weight_chunked_amd import block, ttt_mlp as tm  # noqa: E402


class Block:
    """d_model d, d_ff f, `heads` query heads over `kv_heads` key / value heads of d / heads."""

    def __init__(self, d=256, f=512, heads=4, kv_heads=2, chunk=64, conv_k=4, eta=1e-2,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator()
        g.manual_seed(seed)

        def w(*shape, fan_in):
            return (torch.randn(shape, generator=g) * fan_in ** -0.5).to(dtype).to(device)

        self.d, self.f, self.heads, self.kv_heads, self.dk = d, f, heads, kv_heads, d // heads
        self.chunk, self.eta, self.dtype, self.device = chunk, eta, dtype, device
        width = (heads + 2 * kv_heads) * self.dk
        self.norm1 = torch.ones(d, dtype=dtype, device=device)
        self.norm2 = torch.ones(d, dtype=dtype, device=device)
        self.w_qkv, self.w_o = w(d, width, fan_in=d), w(d, d, fan_in=d)
        self.w_gate, self.w_up = w(f, d, fan_in=d), w(f, d, fan_in=d)
        self.w_down, self.w_target = w(d, f, fan_in=f), w(d, d, fan_in=d)
        self.taps = w(d, conv_k, fan_in=conv_k)
        # memories of two to some hundred tokens
        i = torch.arange(heads, dtype=torch.float32, device=device)
        self.log_decay = -torch.exp2(-1.0 - 7.0 * (i + 0.5) / heads)

    def _ttt(self):
        return self.w_gate, self.w_up, self.w_down, self.taps, self.w_target

    def _split(self, p):
        """q, k, v as views of one projection's rows [B][T][(H + 2 G) dk]."""
        h, g, dk = self.heads, self.kv_heads, self.dk
        return (p[..., :h * dk].unflatten(-1, (h, dk)),
                p[..., h * dk:(h + g) * dk].unflatten(-1, (g, dk)),
                p[..., (h + g) * dk:].unflatten(-1, (g, dk)))

    def mix(self, x, res, state=None, state_out=None):
        """Everything in front of the layer: (h, r, state, what the backward needs)."""
        B, T, d = x.shape
        y, r1, _ = block.add_rmsnorm(x, res, self.norm1)
        raw = (y.view(-1, d) @ self.w_qkv).view(B, T, -1)
        p = raw.clone()
        qk = p[..., :(self.heads + self.kv_heads) * self.dk]
        qk.copy_(torch.nn.functional.silu(qk.float()))
        q, k, v = self._split(p)
        o, state = block.linattn_forward(q, k, v, self.log_decay, state=state,
                                         state_out=state_out)
        a = (o.view(-1, d) @ self.w_o).view(B, T, d)
        h, r2, _ = block.add_rmsnorm(a, r1, self.norm2)
        return h, r2, state, (y, r1, raw, p, o, state)

    def forward(self, x, res, x0):
        """A whole sequence: (out, residual)."""
        h, r, _, _ = self.mix(x, res)
        out, _ = tm.forward_batched(h, x0, *self._ttt(), self.eta, self.chunk)
        return out, r

    def step(self, x, res, x0, dout, lr=0.0):
        """One training step for the loss <dout, out>: gradients of the block's inputs and
        weights; with lr > 0 the weights take an SGD step."""
        B, T, d = x.shape
        h, r2, _, (y, r1, raw, p, o, _) = self.mix(x, res)
        g = tm.backward_batched(h, x0, *self._ttt(), self.eta, self.chunk, dout)
        # the second norm; its sum's gradient is the first part's and the residual's
        dr2, _, dn2 = block.add_rmsnorm_backward(g["H"], r2, self.norm2)
        da = dr2.view(-1, d)
        dw_o = o.view(-1, d).t() @ da
        do = (da @ self.w_o.t()).view_as(o)
        q, k, v = self._split(p)
        ga = block.linattn_backward(q, k, v, self.log_decay, do)
        dp = torch.cat([ga["q"].flatten(2), ga["k"].flatten(2), ga["v"].flatten(2)], -1)
        n = (self.heads + self.kv_heads) * self.dk
        z = raw[..., :n].float()
        s = torch.sigmoid(z)
        dp[..., :n].copy_(dp[..., :n].float() * s * (1 + z * (1 - s)))
        dp = dp.view(-1, dp.shape[-1])
        dw_qkv = y.view(-1, d).t() @ dp
        dy = (dp @ self.w_qkv.t()).view(B, T, d)
        dr1, dx, dn1 = block.add_rmsnorm_backward(dy, r1, self.norm1, dr=dr2)
        grads = {"x": dx, "res": dr1, "norm1": dn1, "norm2": dn2, "w_qkv": dw_qkv, "w_o": dw_o,
                 "w_gate": g["W_gate"], "w_up": g["W_up"], "w_down": g["W_start"].sum(0),
                 "w_target": g["W_target"], "taps": g["taps"]}
        if lr:
            for name, dw in grads.items():
                if name not in ("x", "res"):
                    w = getattr(self, name)
                    w.copy_(w.float() - lr * dw.float())
        return grads


class Session:
    """Sessions served in pieces: the attention's state and the layer's stream."""

    def __init__(self, blk: Block, batch: int):
        self.blk = blk
        self.state = torch.zeros((batch, blk.heads, blk.dk, blk.dk), dtype=torch.float32,
                                 device=blk.device)
        self.stream = tm.Stream(*blk._ttt(), blk.eta, blk.chunk, batch, device=blk.device)

    def feed(self, x, res, x0, last=False):
        h, r, _, _ = self.blk.mix(x, res, self.state, self.state)
        return self.stream.step(h, x0, last=last), r


def main(batch=2, prompt=200, tokens=5):
    g = torch.Generator()
    g.manual_seed(1)
    T = prompt + tokens
    blk = Block()
    x, res, x0, dout = ((torch.randn((batch, T, blk.d), generator=g)).to(blk.dtype).cuda()
                        for _ in range(4))
    out, r = blk.forward(x, res, x0)

    ses, parts = Session(blk, batch), []
    for a, b in [(0, prompt)] + [(t, t + 1) for t in range(prompt, T)]:
        o, _ = ses.feed(*(t[:, a:b].contiguous() for t in (x, res, x0)))
        parts.append(o)
    served = torch.cat(parts, 1)
    err = float((served.float() - out.float()).norm() / out.float().norm())
    print(f"prompt of {prompt} tokens and {tokens} single ones against one call: {err:.2e}")

    before = float((out.float() * dout.float()).sum())
    blk.step(x, res, x0, dout, lr=1e-5)
    after = float((blk.forward(x, res, x0)[0].float() * dout.float()).sum())
    print(f"loss before and after a training step: {before:.3f}, {after:.3f}")
    return err, before, after


if __name__ == "__main__":
    main()
