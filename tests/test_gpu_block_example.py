"""The example block (examples/block.py), which runs the operators together with
the TTT-MLP layer: serving in pieces gives the one-call outputs, and the training
step's gradients are those of the formulas in 64 bits."""
import importlib.util
import os

import pytest
import torch

from chunk_wise_weight_chunked_amd import ttt_mlp as tm

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "block.py")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tm.load()
    spec = importlib.util.spec_from_file_location("example_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_serves_and_trains(ex):
    err, before, after = ex.main()
    # bf16 along the way: some ten roundings of 2^-9 each
    assert err <= 2e-2
    assert after < before


def reference_loss(b, p, x, res, x0, dout):
    """<dout, out> of the block in float64 from its formulas, the layer's chunks one by one."""
    def norm(r, w):
        return r / (r.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w

    B, T, d = x.shape
    H, G, dk = b.heads, b.kv_heads, b.dk
    r1 = x + res
    z = norm(r1, p["norm1"]) @ p["w_qkv"]
    qk = torch.nn.functional.silu(z[..., :(H + G) * dk])
    q = qk[..., :H * dk].reshape(B, T, H, dk)
    k = qk[..., H * dk:].reshape(B, T, G, dk).repeat_interleave(H // G, 2)
    v = z[..., (H + G) * dk:].reshape(B, T, G, dk).repeat_interleave(H // G, 2)
    t = torch.arange(T, dtype=torch.float64)
    dist = t[:, None] - t[None, :]
    w = torch.where(dist >= 0, (b.log_decay.cpu().double()[:, None, None] * dist).exp(), 0.0)
    s = torch.einsum("bthd,bshd->bhts", q, k) * w
    o = torch.einsum("bhts,bshd->bthd", s, v) * dk ** -0.5
    h = norm(r1 + o.reshape(B, T, d) @ p["w_o"], p["norm2"])
    Z = torch.nn.functional.silu(h @ p["w_gate"].T) * (h @ p["w_up"].T)
    pad = torch.cat([x0, torch.zeros(B, 8, d, dtype=x0.dtype)], 1)
    front = torch.cat([torch.zeros(B, 8, d, dtype=x0.dtype), pad], 1)
    U = sum(p["taps"][:, i] * front[:, 8 + 1 - i:8 + 1 - i + T] for i in range(p["taps"].shape[1]))
    V = U @ p["w_target"]
    W, out = p["w_down"].expand(B, -1, -1), []
    for a in range(0, T, b.chunk):
        e = min(a + b.chunk, T)
        out.append(Z[:, a:e] @ W.transpose(1, 2))
        W = W + b.eta * V[:, a:e].transpose(1, 2) @ Z[:, a:e]
    return (torch.cat(out, 1) * dout).sum()


def test_training_step_gradients(ex):
    b = ex.Block(d=128, f=192, heads=4, kv_heads=2, chunk=32)
    g = torch.Generator()
    g.manual_seed(3)
    B, T = 2, 75
    x, res, x0, dout = (torch.randn((B, T, b.d), generator=g).to(b.dtype).cuda() for _ in range(4))
    got = b.step(x, res, x0, dout)
    names = ["norm1", "norm2", "w_qkv", "w_o", "w_gate", "w_up", "w_down", "w_target", "taps"]
    p = {n: getattr(b, n).cpu().double().requires_grad_(True) for n in names}
    xs = [t.cpu().double().requires_grad_(True) for t in (x, res)]
    loss = reference_loss(b, p, *xs, x0.cpu().double(), dout.cpu().double())
    want = dict(zip(["x", "res"] + names, torch.autograd.grad(loss, xs + list(p.values()))))
    for n, w in want.items():
        e = float((got[n].cpu().double() - w).norm() / w.norm())
        print(n, "%.2e" % e, flush=True)
        assert e <= 3e-2, (n, e)  # the layer's own bound (2e-2) and the block's roundings
