"""From token ids through a block and back, with this library's operators: a prompt, the tokens
after it, and one training step that keeps its activations in 8 bits.

    python examples/stack.py

    e = table[ids] * scale                 embed_forward: the residual stream and the layer's X0
    y = norm(e)                            add_rmsnorm
    x, gates = y W_in                      the caller's matrix product
    h = gated recurrence of x              gatedrec_forward, one fp32 state a channel and session
    r = e + h W_o, z = norm(r)             add_rmsnorm
    out = TTT-MLP(z, X0 = e)               ttt_mlp.forward_batched / Stream

Trained, the weight gradients of W_in and W_o come from y and h as act8_store keeps them, the
recurrence's inputs are read back by act8_load, and the embeddings' gradient (from the residual
stream and from the layer's X0) goes to the table by embed_backward.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from chunk_wise_weight_chunked_amd import block, seq, ttt_mlp as tm  # noqa: E402


class Stack:
    """`vocab` tokens, d_model d, d_ff f."""

    def __init__(self, vocab=1000, d=256, f=512, chunk=64, conv_k=4, eta=1e-2,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator()
        g.manual_seed(seed)

        def w(*shape, fan_in):
            return (torch.randn(shape, generator=g) * fan_in ** -0.5).to(dtype).to(device)

        self.vocab, self.d, self.f, self.chunk, self.eta = vocab, d, f, chunk, eta
        self.dtype, self.device, self.scale = dtype, device, d ** 0.5
        self.table = w(vocab, d, fan_in=d)
        self.norm1 = torch.ones(d, dtype=dtype, device=device)
        self.norm2 = torch.ones(d, dtype=dtype, device=device)
        self.w_in, self.w_o = w(d, 3 * d, fan_in=d), w(d, d, fan_in=d)
        # memories of about one to some hundred tokens
        self.rate = torch.exp(4.0 * torch.rand(d, generator=g) - 4.0).to(device)
        self.w_gate, self.w_up = w(f, d, fan_in=d), w(f, d, fan_in=d)
        self.w_down, self.w_target = w(d, f, fan_in=f), w(d, d, fan_in=d)
        self.taps = w(d, conv_k, fan_in=conv_k)

    def _ttt(self):
        return self.w_gate, self.w_up, self.w_down, self.taps, self.w_target

    def mix(self, ids, state=None, state_out=None, save=False):
        """Everything in front of the layer: (z, e, what the backward needs)."""
        B, T = ids.shape
        d = self.d
        e = seq.embed_forward(ids, self.table, self.scale)
        y, _, _ = block.add_rmsnorm(e, None, self.norm1)
        p = (y.view(-1, d) @ self.w_in).view(B, T, 3 * d)
        h, _, saved = seq.gatedrec_forward(p[..., :d], p[..., d:2 * d], p[..., 2 * d:], self.rate,
                                           state=state, state_out=state_out, save=save)
        a = (h.view(-1, d) @ self.w_o).view(B, T, d)
        z, r, _ = block.add_rmsnorm(a, e, self.norm2)
        return z, e, (y, p, h, saved, r)

    def forward(self, ids):
        """Whole sequences [B][T]: the layer's outputs [B][T][d]."""
        z, e, _ = self.mix(ids)
        return tm.forward_batched(z, e, *self._ttt(), self.eta, self.chunk)[0]

    def step(self, ids, dout, keep8=True):
        """Gradients of the weights for the loss <dout, out>; with keep8 the activations between
        the forward and the backward pass are held in 8 bits."""
        B, T = ids.shape
        d = self.d
        z, e, (y, p, h, saved, r) = self.mix(ids, save=True)
        if keep8:
            y8, p8, h8 = seq.act8_store(y), seq.act8_store(p), seq.act8_store(h)
            del y, p, h
        g = tm.backward_batched(z, e, *self._ttt(), self.eta, self.chunk, dout)
        dr, _, dn2 = block.add_rmsnorm_backward(g["H"], r, self.norm2)
        dh = (dr.view(-1, d) @ self.w_o.t()).view(B, T, d)
        if keep8:
            dw_o = seq.act8_weight_grad(*h8, dr)
            p = seq.act8_load(*p8, dtype=self.dtype)
        else:
            dw_o = h.view(-1, d).t() @ dr.view(-1, d)
        ga = seq.gatedrec_backward(p[..., :d], p[..., d:2 * d], p[..., 2 * d:], self.rate, dh,
                                   saved)
        dp = torch.cat([ga["x"], ga["decay_gate"], ga["input_gate"]], -1)
        dw_in = (seq.act8_weight_grad(*y8, dp) if keep8
                 else y.view(-1, d).t() @ dp.view(-1, 3 * d))
        dy = (dp.view(-1, 3 * d) @ self.w_in.t()).view(B, T, d)
        de, _, dn1 = block.add_rmsnorm_backward(dy, e, self.norm1, dr=dr)
        de = (de.float() + g["X0"].float()).to(self.dtype)
        return {"table": seq.embed_backward(de, ids, self.vocab, self.scale),
                "norm1": dn1, "norm2": dn2, "w_in": dw_in, "w_o": dw_o, "rate": ga["rate"],
                "w_gate": g["W_gate"], "w_up": g["W_up"], "w_down": g["W_start"].sum(0),
                "w_target": g["W_target"], "taps": g["taps"]}


class Session:
    """Sessions served in pieces: the recurrence's state and the layer's stream."""

    def __init__(self, stack: Stack, batch: int):
        self.stack = stack
        self.state = torch.zeros((batch, stack.d), dtype=torch.float32, device=stack.device)
        self.stream = tm.Stream(*stack._ttt(), stack.eta, stack.chunk, batch, device=stack.device)

    def feed(self, ids, last=False):
        z, e, _ = self.stack.mix(ids, self.state, self.state)
        return self.stream.step(z, e, last=last)


def main(batch=2, prompt=200, tokens=5):
    g = torch.Generator()
    g.manual_seed(1)
    T = prompt + tokens
    stack = Stack()
    ids = torch.randint(0, stack.vocab, (batch, T), generator=g).cuda()
    out = stack.forward(ids)

    ses, parts = Session(stack, batch), []
    for a, b in [(0, prompt)] + [(t, t + 1) for t in range(prompt, T)]:
        parts.append(ses.feed(ids[:, a:b].contiguous()))
    served = torch.cat(parts, 1)
    err = float((served.float() - out.float()).norm() / out.float().norm())
    print(f"prompt of {prompt} tokens and {tokens} single ones against one call: {err:.2e}")

    dout = torch.randn(out.shape, generator=g).to(out.dtype).cuda()
    off = {}
    full, kept = stack.step(ids, dout, keep8=False), stack.step(ids, dout)
    for n in full:
        off[n] = float((kept[n].float() - full[n].float()).norm() / full[n].float().norm())
    print("gradients with activations kept in 8 bits, off by: "
          + ", ".join(f"{n} {e:.1e}" for n, e in off.items()))
    return err, off


if __name__ == "__main__":
    main()
