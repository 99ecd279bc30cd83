"""Pins of oracle/train.py: values against loops over single numbers, gradients against
central differences of the function they belong to, and the whole layer against a dense
form that knows no rows."""

import math

import pytest
import torch

from oracle import train as ot
from oracle.block import act_ref
from oracle.moe import plan_ref

F64 = torch.float64
ACTS = ["none", "relu", "silu", "gelu", "sigmoid"]


def _rand(*shape, seed, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * scale


def _differences(fun, x, step=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        hi, lo = x.clone(), x.clone()
        hi.view(-1)[i] += step
        lo.view(-1)[i] -= step
        g.view(-1)[i] = (float(fun(hi)) - float(fun(lo))) / (2 * step)
    return g


IDS = torch.tensor([[1, 0], [2, -1], [1, 2], [-1, 9], [0, 0]], dtype=torch.int32)    # 9 of 10 picks in 0..2, dropped ones
T, K, E = 5, 2, 3


@pytest.fixture(scope="module")
def plan():
    p = plan_ref(IDS.numpy(), E)
    return torch.from_numpy(p["pair_rows"]), torch.from_numpy(p["expert_offsets"])


def test_rows_and_back_by_loops_and_differences(plan):
    pair_rows, off = plan
    live = int(off[-1])
    assert live == 7
    x, w, add, dy = _rand(T, 4, seed=1), _rand(T, K, seed=2), _rand(T, 4, seed=3), _rand(T, 4, seed=4)
    rows = torch.zeros(T * K, 4, dtype=F64)
    seen = ot.sort_rows_ref(x, pair_rows, T, K)
    assert sorted(seen) == list(range(live))
    for r, v in seen.items():
        rows[r] = v
        e = int(torch.searchsorted(off, torch.tensor(r, dtype=off.dtype), right=True)) - 1
        assert any(torch.equal(v, x[t]) and e in IDS[t].tolist() for t in range(T))
    y, mag = ot.return_rows_ref(rows, pair_rows, T, K, w, add)
    for t in range(T):
        for c in range(4):
            want = float(add[t, c]) + sum(float(w[t, j]) * float(x[t, c]) for j in range(K) if 0 <= int(IDS[t, j]) < E)
            assert float(y[t, c]) == pytest.approx(want, rel=1e-13) and float(mag[t, c]) >= abs(want) * (1 - 1e-13)
    rows = _rand(T * K, 4, seed=5)
    d_rows, d_w, _ = ot.return_rows_grad_ref(dy, rows, pair_rows, T, K, w)
    loss = lambda r, v: (ot.return_rows_ref(r, pair_rows, T, K, v, add)[0] * dy).sum()  # noqa: E731
    assert torch.allclose(d_w, _differences(lambda v: loss(rows, v), w), atol=1e-8)
    want = _differences(lambda r: loss(r, w), rows)
    for r in range(T * K):
        assert torch.allclose(d_rows.get(r, torch.zeros(4, dtype=F64)), want[r], atol=1e-8)
    # the gradient of laying rows out is bringing them back
    up = _rand(T * K, 4, seed=6)
    laid = lambda v: sum((ot.sort_rows_ref(v, pair_rows, T, K)[r] * up[r]).sum() for r in range(live))  # noqa: E731
    assert torch.allclose(ot.return_rows_ref(up, pair_rows, T, K)[0], _differences(laid, x), atol=1e-8)


def test_products_by_loops_and_differences(plan):
    off = plan[1]
    x, w, dy = _rand(T * K, 3, seed=1), _rand(E + 1, 2, 3, seed=2), _rand(T * K, 2, seed=3)
    off = torch.cat([off, off[-1:]])                       # a fourth expert without rows
    y, mag = ot.expert_linear_ref(x, w, off)
    for r in range(T * K):
        e = next((e for e in range(E + 1) if off[e] <= r < off[e + 1]), None)
        for n in range(2):
            terms = [] if e is None else [float(x[r, c]) * float(w[e, n, c]) for c in range(3)]
            assert float(y[r, n]) == pytest.approx(math.fsum(terms), rel=1e-12, abs=1e-15)
            assert float(mag[r, n]) == pytest.approx(math.fsum(abs(v) for v in terms), rel=1e-12)
    loss = lambda a, b: (ot.expert_linear_ref(a, b, off)[0] * dy).sum()  # noqa: E731
    dx, dw, mx, mw = ot.expert_linear_grad_ref(dy, x, w, off)
    assert torch.allclose(dx, _differences(lambda v: loss(v, w), x), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda v: loss(x, v), w), atol=1e-8)
    assert bool((dw[E] == 0).all()) and bool((mx >= dx.abs() - 1e-12).all()) and bool((mw >= dw.abs() - 1e-12).all())


@pytest.mark.parametrize("act", ACTS)
def test_glu_by_loops_and_differences(act):
    z, dh = _rand(3, 8, seed=1), _rand(3, 4, seed=2)
    h = ot.glu_ref(z, act)
    for r in range(3):
        for c in range(4):
            g, u = float(z[r, c]), float(z[r, 4 + c])
            a = {"none": g, "relu": max(g, 0.0), "silu": g / (1 + math.exp(-g)), "sigmoid": 1 / (1 + math.exp(-g)),
                 "gelu": g * 0.5 * (1 + math.erf(g / math.sqrt(2)))}[act]
            assert float(h[r, c]) == pytest.approx(a * u, rel=1e-12)
    dz, again = ot.glu_grad_ref(dh, z, act)
    assert torch.equal(again, h)
    assert torch.allclose(dz, _differences(lambda v: (ot.glu_ref(v, act) * dh).sum(), z), atol=1e-8)


def test_saved_values_are_the_nearest():
    z = _rand(4, 256, seed=1, scale=3.0)
    z[2, :128] = 0
    q, s = ot.saved_ref(z)
    v = ot.restored_ref(q, s)
    step = torch.exp2(s.to(F64) - 127).repeat_interleave(128, 1)
    assert bool(((v - z).abs() <= torch.maximum(z.abs() * 2.0 ** -4, step * 2.0 ** -10)).all())
    assert bool((v[2, :128] == 0).all())
    top = z.abs().view(4, 2, 128).amax(2)
    assert bool((top <= 448 * step[:, ::128]).all()) and bool(((top > 224 * step[:, ::128]) | (top == 0)).all())


def test_the_layer_is_the_dense_one(plan):
    """Rows, products, activation and return against every expert on every token."""
    pair_rows, off = plan
    x, w13, w2, wt = _rand(T, 4, seed=1), _rand(E, 6, 4, seed=2), _rand(E, 4, 3, seed=3), _rand(T, K, seed=4)
    rows = torch.zeros(T * K, 4, dtype=F64)
    for r, v in ot.sort_rows_ref(x, pair_rows, T, K).items():
        rows[r] = v
    h = ot.glu_ref(ot.expert_linear_ref(rows, w13, off)[0], "silu")
    y = ot.return_rows_ref(ot.expert_linear_ref(h, w2, off)[0], pair_rows, T, K, wt)[0]
    want = torch.zeros(T, 4, dtype=F64)
    for t in range(T):
        for j in range(K):
            e = int(IDS[t, j])
            if 0 <= e < E:
                z = w13[e] @ x[t]
                want[t] += wt[t, j] * (w2[e] @ (act_ref(z[:3], "silu") * z[3:]))
    assert torch.allclose(y, want, rtol=1e-12, atol=1e-12)
