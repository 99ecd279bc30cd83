"""Training the experts in float64: rows by expert and back, the experts' products, the
gated activation with its input saved in 8 bits, and their gradients. torch CPU tensors
in, float64 out, written from the definitions with loops over pairs and experts (pinned
by tests/test_oracle_train.py against differences and a dense form)."""

from __future__ import annotations

import torch

from .block import F64, act_ref, act_slope_ref
from .formats import dequantize_blocks, quantize_blocks


def sort_rows_ref(x, pair_rows, T, K):
    """{row: values} of every pick that was not dropped."""
    x = x.to(F64)
    return {int(r): x[p // K] for p, r in enumerate(pair_rows[:T * K].tolist()) if r >= 0}


def return_rows_ref(rows, pair_rows, T, K, weights=None, add=None):
    """(y, magnitude): the sum of weighted rows plus add, and of the terms' absolute values."""
    H = rows.shape[1]
    y = torch.zeros(T, H, dtype=F64) if add is None else add.to(F64).clone()
    mag = y.abs()
    for p, r in enumerate(pair_rows[:T * K].tolist()):
        if r >= 0:
            v = rows[r].to(F64) * (1.0 if weights is None else float(weights[p // K, p % K]))
            y[p // K] += v
            mag[p // K] += v.abs()
    return y, mag


def return_rows_grad_ref(dy, rows, pair_rows, T, K, weights=None):
    """({row: d_rows}, d_weights, magnitude of d_weights' terms)."""
    dy = dy.to(F64)
    d_rows, dw, mag = {}, torch.zeros(T, K, dtype=F64), torch.zeros(T, K, dtype=F64)
    for p, r in enumerate(pair_rows[:T * K].tolist()):
        t, j = p // K, p % K
        if r >= 0:
            d_rows[r] = dy[t] * (1.0 if weights is None else float(weights[t, j]))
            terms = rows[r].to(F64) * dy[t]
            dw[t, j], mag[t, j] = terms.sum(), terms.abs().sum()
    return d_rows, dw, mag


def expert_linear_ref(x, w, offsets):
    """(y, magnitude); rows of no expert are zero."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=F64)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            a, b = x[lo:hi].to(F64), w[e].to(F64).t()
            y[lo:hi], mag[lo:hi] = a @ b, a.abs() @ b.abs()
    return y, mag


def expert_linear_grad_ref(dy, x, w, offsets):
    """(dx, dw, magnitudes of both)."""
    dx, dw = torch.zeros(x.shape, dtype=F64), torch.zeros(w.shape, dtype=F64)
    mx, mw = torch.zeros_like(dx), torch.zeros_like(dw)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            d, a, b = dy[lo:hi].to(F64), x[lo:hi].to(F64), w[e].to(F64)
            dx[lo:hi], mx[lo:hi] = d @ b, d.abs() @ b.abs()
            dw[e], mw[e] = d.t() @ a, d.abs().t() @ a.abs()
    return dx, dw, mx, mw


def saved_ref(z):
    """(codes, scales) uint8 of z's columns in blocks of 128."""
    q, s, _ = quantize_blocks(z.to(F64).numpy())
    return torch.from_numpy(q), torch.from_numpy(s)


def restored_ref(q, s):
    """What codes and scales stand for."""
    return torch.from_numpy(dequantize_blocks(q.numpy(), s.numpy()))


def glu_ref(z, act):
    z = z.to(F64)
    I = z.shape[1] // 2
    return act_ref(z[:, :I], act) * z[:, I:]


def glu_grad_ref(dh, z, act):
    """(dz, h) at z."""
    z, dh = z.to(F64), dh.to(F64)
    I = z.shape[1] // 2
    g, u = z[:, :I], z[:, I:]
    a = act_ref(g, act)
    return torch.cat([dh * u * act_slope_ref(g, act), dh * a], 1), a * u
