"""The operators in front of the FFN in float64: residual add + RMS norm, dense product
with its epilogue, gate, balance loss, and their gradients. torch CPU tensors in,
float64 out, written from the definitions (pinned by tests/test_oracle_block.py against
loops and finite differences)."""

from __future__ import annotations

import math

import torch

F64 = torch.float64
SUM_EPS = 1e-20


def add_norm_ref(x, weight, residual=None, eps=1e-6):
    """(h, y): h = x + residual; y = weight * h / sqrt(mean(h^2) + eps)."""
    h = x.to(F64)
    if residual is not None:
        h = h + residual.to(F64)
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * weight.to(F64)


def add_norm_grad_ref(dy, h, weight, eps=1e-6, dh=None):
    """(dx, dweight) of add_norm_ref at h."""
    dy, h, w = dy.to(F64), h.to(F64), weight.to(F64)
    H = h.shape[1]
    var = (h * h).mean(1, keepdim=True) + eps
    g = dy * w
    dx = g / var.sqrt() - h * (g * h).sum(1, keepdim=True) / (H * var * var.sqrt())
    if dh is not None:
        dx = dx + dh.to(F64)
    return dx, (dy * h / var.sqrt()).sum(0)


def act_ref(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    assert act == "none"
    return z


def act_slope_ref(z, act):
    p = 1 / (1 + torch.exp(-z))
    if act == "relu":
        return (z > 0).to(F64)
    if act == "silu":
        return p + z * p * (1 - p)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        return p * (1 - p)
    return torch.ones_like(z)


def linear_ref(x, w, bias=None, act="none", residual=None):
    """(y, z): z = x w^T + bias, y = act(z) + residual."""
    z = x.to(F64) @ w.to(F64).t()
    if bias is not None:
        z = z + bias.to(F64)
    y = act_ref(z, act)
    return (y if residual is None else y + residual.to(F64)), z


def linear_grad_ref(dy, x, w, act="none", z=None):
    """(dx, dw, dbias, dz) of linear_ref."""
    dz = dy.to(F64)
    if act != "none":
        dz = dz * act_slope_ref(z.to(F64), act)
    return dz @ w.to(F64), dz.t() @ x.to(F64), dz.sum(0), dz


def clean_logits(l):
    """float64 logits with NaN masked and +inf as the largest float32."""
    l = l.to(F64)
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    return l.clamp(max=torch.finfo(torch.float32).max)


def scores_ref(l, score):
    """Scores of clean logits; masked experts score 0."""
    dead = l == -math.inf
    if score == "softmax":
        top = torch.where(dead, torch.full_like(l, -1e300), l).amax(1, keepdim=True)
        e = torch.where(dead, torch.zeros_like(l), torch.exp(l - top))
        total = e.sum(1, keepdim=True)
        return torch.where(total > 0, e / total.clamp(min=1e-300), torch.zeros_like(l))
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        assert score == "sqrtsoftplus"
        s = torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))
    return torch.where(dead, torch.zeros_like(l), s)


def score_slope_ref(l, s, score):
    dead = l == -math.inf
    p = 1 / (1 + torch.exp(-l))
    d = s * (1 - p) if score == "sigmoid" else p / (2 * s).clamp(min=1e-300)
    return torch.where(dead, torch.zeros_like(l), d)


def gate_ref(logits, K, score="softmax", bias=None, renorm=True, scale=1.0, n_valid=None):
    """(ids, weights) as lists over rows: the K experts of the largest score + bias,
    equal ones by ascending index; -1 and weight 0 where there is none."""
    l = clean_logits(logits)
    T, E = l.shape
    s = scores_ref(l, score)
    ids = torch.full((T, K), -1, dtype=torch.int32)
    w = torch.zeros((T, K), dtype=F64)
    for t in range(T if n_valid is None else max(0, min(T, n_valid))):
        key = l[t] if bias is None else s[t] + bias.to(F64)
        ok = [e for e in range(E) if l[t, e] > -math.inf and key[e] > -math.inf]
        order = sorted(ok, key=lambda e: (-float(key[e]), e))[:K]
        for j, e in enumerate(order):
            ids[t, j] = e
            w[t, j] = s[t, e]
    if renorm:
        w = w / (w.sum(1, keepdim=True) + SUM_EPS)
    return ids, w * scale


def gate_grad_ref(logits, ids, d_weights, score="softmax", renorm=True, scale=1.0, add=None):
    """(d_logits, magnitude): the gradient, and the sum of the absolute values of the
    terms it adds up (what its rounding errors are relative to)."""
    l = clean_logits(logits)
    T, E = l.shape
    s = scores_ref(l, score)
    ok = (ids >= 0) & (ids < E)
    at = torch.where(ok, ids, torch.zeros_like(ids)).long()
    c = torch.where(ok, s.gather(1, at), torch.zeros(1, dtype=F64))
    dw = torch.where(ok, d_weights.to(F64), torch.zeros(1, dtype=F64))
    if renorm:
        S = c.sum(1, keepdim=True) + SUM_EPS
        dc, mag = scale * (dw - (dw * c).sum(1, keepdim=True) / S) / S, scale * (dw.abs() + (dw.abs() * c).sum(1, keepdim=True) / S) / S
    else:
        dc = scale * dw
        mag = dc.abs()
    zero = torch.zeros(1, dtype=F64)
    ds = torch.zeros(T, E, dtype=F64).scatter_add_(1, at, torch.where(ok, dc, zero))
    dm = torch.zeros(T, E, dtype=F64).scatter_add_(1, at, torch.where(ok, mag, zero))
    if score == "softmax":
        dl, m = s * (ds - (ds * s).sum(1, keepdim=True)), s * (dm + (dm * s).sum(1, keepdim=True))
    else:
        k = score_slope_ref(l, s, score)
        dl, m = ds * k, dm * k
    if add is not None:
        dl, m = dl + add.to(F64), m + add.to(F64).abs()
    return dl, m


def balance_loss_ref(logits, ids, alpha, score="softmax", seq_offsets=None):
    """(loss, counts, d_logits, magnitude)."""
    l = clean_logits(logits)
    T, E = l.shape
    K = ids.shape[1]
    s = scores_ref(l, score)
    total = s.sum(1, keepdim=True)
    p = torch.where(total > 0, s / total.clamp(min=1e-300), torch.zeros_like(s))
    off = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    B = len(off) - 1
    counts = torch.zeros(B, E, dtype=torch.int32)
    dl, mag = torch.zeros(T, E, dtype=F64), torch.zeros(T, E, dtype=F64)
    loss = 0.0
    for b in range(B):
        lo, hi = off[b], off[b + 1]
        if hi <= lo:
            continue
        n = hi - lo
        for e in ids[lo:hi].reshape(-1).tolist():
            if 0 <= e < E:
                counts[b, e] += 1
        f = counts[b].to(F64) * E / (K * n)
        pb = p[lo:hi]
        loss += alpha / B * float((f * pb.mean(0)).sum())
        a = alpha / B / n * f
        dot = (pb * a).sum(1, keepdim=True)
        if score == "softmax":
            k = pb
        else:
            k = torch.where(total[lo:hi] > 0, score_slope_ref(l[lo:hi], s[lo:hi], score) / total[lo:hi].clamp(min=1e-300),
                            torch.zeros_like(pb))
        dl[lo:hi], mag[lo:hi] = k * (a - dot), k * (a + dot).abs()
    return loss, counts, dl, mag
