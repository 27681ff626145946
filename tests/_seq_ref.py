"""Plain 64-bit forms of the sequence operators on the CPU, from their definitions,
for the tests: one token after the other, one group after the other."""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def embed_grad(dout, ids, vocab, scale, start=None):
    """dout [N][d], ids [N] -> grad [vocab][d] in float64."""
    g = np.zeros((vocab, dout.shape[1])) if start is None else start.astype(np.float64).copy()
    ok = (ids >= 0) & (ids < vocab)
    np.add.at(g, ids[ok], scale * dout[ok])
    return g


def gatedrec(x, dg, ig, rate, state=None, lengths=None):
    """x, dg, ig [B][T][d], rate [d] in float64 -> (h, final state)."""
    B, T, d = x.shape
    h = np.zeros((B, T, d))
    S = np.zeros((B, d)) if state is None else state.copy()
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for t in range(n):
            z = -rate * sigmoid(dg[b, t])
            S[b] = np.exp(z) * S[b] + np.sqrt(-np.expm1(2 * z)) * sigmoid(ig[b, t]) * x[b, t]
            h[b, t] = S[b]
    return h, S


def gatedrec_grads(x, dg, ig, rate, dh, state=None, dstate=None, lengths=None):
    """Gradients of <dh, h> + <dstate, final state>: dx, ddecay, dinput, drate, dstate_in."""
    B, T, d = x.shape
    h, _ = gatedrec(x, dg, ig, rate, state, lengths)
    dx, ddg, dig = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    drate, ds = np.zeros(d), np.zeros((B, d))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        c = np.zeros(d) if dstate is None else dstate[b].copy()
        for t in range(n - 1, -1, -1):
            r, i = sigmoid(dg[b, t]), sigmoid(ig[b, t])
            z = -rate * r
            a, bb = np.exp(z), np.sqrt(-np.expm1(2 * z))
            before = h[b, t - 1] if t else (0.0 if state is None else state[b])
            lam = dh[b, t] + c
            dx[b, t] = lam * bb * i
            dig[b, t] = lam * bb * x[b, t] * i * (1 - i)
            slope = np.divide(a * a, bb, out=np.zeros_like(bb), where=bb > 0)
            dz = lam * (a * before - i * x[b, t] * slope)
            ddg[b, t] = dz * -rate * r * (1 - r)
            drate -= dz * r
            c = a * lam
        ds[b] = c
    return dx, ddg, dig, drate, ds


def act8(x):
    """x [rows][d] float64 -> (codes, exps): each group of 32 by its largest value."""
    rows, d = x.shape
    codes = np.zeros((rows, d), np.int8)
    exps = np.zeros((rows, -(-d // 32)), np.uint8)
    for r in range(rows):
        for g in range(exps.shape[1]):
            v = x[r, 32 * g:32 * g + 32]
            if not np.isfinite(v).all():
                exps[r, g] = 255
                continue
            e = -126
            while np.abs(v).max() > 127 * 2.0 ** e and e < 121:
                e += 1
            exps[r, g] = e + 127
            codes[r, 32 * g:32 * g + 32] = np.clip(np.rint(v * 2.0 ** -e), -127, 127)
    return codes, exps


def act8_value(codes, exps):
    scale = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    return codes.astype(np.float64) * np.repeat(scale, 32, axis=1)[:, :codes.shape[1]]
