"""Plain 64-bit forms of the block operators on the CPU, from their definitions,
for the tests: one token after the other, one row after the other."""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def rel(a, b) -> float:
    a, b = np.asarray(a, np.float64).ravel(), np.asarray(b, np.float64).ravel()
    nb = np.linalg.norm(b)
    d = np.linalg.norm(a - b)
    return float(d / nb) if nb > 0 else float(d)


def linattn(q, k, v, log_decay, scale, state=None, lengths=None):
    """q [B][T][H][dk], k [B][T][G][dk], v [B][T][G][dv] in float64 -> (o, final state)."""
    B, T, H, dk = q.shape
    G, dv = k.shape[2], v.shape[3]
    g = np.exp(log_decay)
    o = np.zeros((B, T, H, dv))
    S = np.zeros((B, H, dk, dv)) if state is None else state.copy()
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for h in range(H):
            kh = h // (H // G)
            for t in range(n):
                S[b, h] = g[h] * S[b, h] + np.outer(k[b, t, kh], v[b, t, kh])
                o[b, t, h] = scale * (q[b, t, h] @ S[b, h])
    return o, S


def linattn_grads(q, k, v, log_decay, scale, dO, state=None, dstate=None, lengths=None):
    """Gradients of <dO, o> + <dstate, final state> by running the recurrence backwards."""
    B, T, H, dk = q.shape
    G, dv = k.shape[2], v.shape[3]
    g = np.exp(log_decay)
    dq, dk_, dv_ = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dS0 = np.zeros((B, H, dk, dv))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for h in range(H):
            kh = h // (H // G)
            S = np.zeros((dk, dv)) if state is None else state[b, h].copy()
            for t in range(n):
                S = g[h] * S + np.outer(k[b, t, kh], v[b, t, kh])
                dq[b, t, h] = scale * (S @ dO[b, t, h])
            D = np.zeros((dk, dv)) if dstate is None else dstate[b, h].copy()
            for t in range(n - 1, -1, -1):
                D = D + scale * np.outer(q[b, t, h], dO[b, t, h])   # gradient of S_t
                dk_[b, t, kh] += D @ v[b, t, kh]
                dv_[b, t, kh] += D.T @ k[b, t, kh]
                D = g[h] * D
            dS0[b, h] = D
    return dq, dk_, dv_, dS0


def addnorm(x, res, w, eps):
    r = x if res is None else x + res
    return r, r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * w


def addnorm_grads(dy, r, w, eps, dr_out=None):
    d = r.shape[-1]
    dx, dw = np.zeros_like(r), np.zeros(d)
    for i in range(r.shape[0]):
        s = 1.0 / np.sqrt((r[i] ** 2).sum() / d + eps)
        # y_j = r_j s w_j, ds/dr_i = -s^3 r_i / d
        dx[i] = dy[i] * w * s - (dy[i] * w * r[i]).sum() * s ** 3 / d * r[i]
        dw += dy[i] * r[i] * s
    return (dx if dr_out is None else dx + dr_out), dw
