"""Pins of oracle/block.py: each function against loops over single numbers, each
gradient against central differences of the function it belongs to."""

import math

import pytest
import torch

from oracle import block as ob

F64 = torch.float64


def _rand(*shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=F64) * scale


def _differences(fun, x, step=1e-5):
    """Central differences of a scalar function at x."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        hi, lo = x.clone(), x.clone()
        hi.view(-1)[i] += step
        lo.view(-1)[i] -= step
        g.view(-1)[i] = (float(fun(hi)) - float(fun(lo))) / (2 * step)
    return g


def test_add_norm_by_loops_and_its_gradient():
    x, res, w, dy, dh = (_rand(3, 8, seed=i) for i in range(5))
    w = w[0]
    h, y = ob.add_norm_ref(x, w, res, eps=0.1)
    for t in range(3):
        row = [float(x[t, i]) + float(res[t, i]) for i in range(8)]
        r = 1 / math.sqrt(math.fsum(v * v for v in row) / 8 + 0.1)
        for i in range(8):
            assert float(h[t, i]) == row[i]
            assert float(y[t, i]) == pytest.approx(row[i] * r * float(w[i]), rel=1e-14)
    dx, dw = ob.add_norm_grad_ref(dy, h, w, eps=0.1, dh=dh)
    loss = lambda hh, ww: (ob.add_norm_ref(hh, ww, eps=0.1)[1] * dy).sum() + (hh * dh).sum()
    torch.testing.assert_close(dx, _differences(lambda v: loss(v, w), h), rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(dw, _differences(lambda v: loss(h, v), w), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "sigmoid"])
def test_linear_by_loops_and_its_gradient(act):
    x, w, b, res, dy = _rand(3, 6, seed=1), _rand(4, 6, seed=2), _rand(4, seed=3), _rand(3, 4, seed=4), _rand(3, 4, seed=5)
    y, z = ob.linear_ref(x, w, b, act, res)
    one = {"none": lambda v: v, "relu": lambda v: max(v, 0.0), "silu": lambda v: v / (1 + math.exp(-v)),
           "gelu": lambda v: v * 0.5 * (1 + math.erf(v / math.sqrt(2))), "sigmoid": lambda v: 1 / (1 + math.exp(-v))}[act]
    for m in range(3):
        for n in range(4):
            v = math.fsum(float(x[m, k]) * float(w[n, k]) for k in range(6)) + float(b[n])
            assert float(z[m, n]) == pytest.approx(v, rel=1e-13)
            assert float(y[m, n]) == pytest.approx(one(v) + float(res[m, n]), rel=1e-12)
    dx, dw, db, _ = ob.linear_grad_ref(dy, x, w, act, z)
    loss = lambda xx, ww, bb: (ob.linear_ref(xx, ww, bb, act, res)[0] * dy).sum()
    torch.testing.assert_close(dx, _differences(lambda v: loss(v, w, b), x), rtol=1e-6, atol=1e-8)
    torch.testing.assert_close(dw, _differences(lambda v: loss(x, v, b), w), rtol=1e-6, atol=1e-8)
    torch.testing.assert_close(db, _differences(lambda v: loss(x, w, v), b), rtol=1e-6, atol=1e-8)


def _score_by_loop(row, e, score):
    if score == "softmax":
        return math.exp(row[e]) / math.fsum(math.exp(v) for v in row)
    if score == "sigmoid":
        return 1 / (1 + math.exp(-row[e]))
    return math.sqrt(math.log(1 + math.exp(row[e])))


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_by_loops_and_its_gradient(score, renorm):
    l, dw, bias, add = _rand(4, 7, seed=6), _rand(4, 3, seed=7), _rand(7, seed=8, scale=0.2), _rand(4, 7, seed=9)
    ids, w = ob.gate_ref(l, 3, score, bias, renorm, 2.5)
    for t in range(4):
        row = l[t].tolist()
        s = [_score_by_loop(row, e, score) for e in range(7)]
        left, picks = list(range(7)), []
        for _ in range(3):
            best = max(left, key=lambda e: s[e] + float(bias[e]))
            picks.append(best)
            left.remove(best)
        assert ids[t].tolist() == picks
        total = sum(s[e] for e in picks) if renorm else 1.0
        assert w[t].tolist() == pytest.approx([2.5 * s[e] / total for e in picks], rel=1e-12)

    def loss(ll):
        s = ob.scores_ref(ll, score).gather(1, ids.long())
        if renorm:
            s = s / (s.sum(1, keepdim=True) + ob.SUM_EPS)
        return (2.5 * s * dw).sum()
    dl, mag = ob.gate_grad_ref(l, ids, dw, score, renorm, 2.5)
    torch.testing.assert_close(dl, _differences(loss, l), rtol=1e-6, atol=1e-8)
    assert bool((mag >= dl.abs() - 1e-15).all())
    torch.testing.assert_close(ob.gate_grad_ref(l, ids, dw, score, renorm, 2.5, add)[0], dl + add)


def test_gate_masks_ties_and_padding():
    inf = math.inf
    l = torch.tensor([[1.0, 2.0, 2.0, -inf, math.nan], [-inf] * 5, [inf, 0.0, inf, 1.0, 2.0], [0.0, 1.0, 2.0, 3.0, 4.0]],
                     dtype=F64)
    ids, w = ob.gate_ref(l, 4, "sigmoid", n_valid=3)
    assert ids.tolist() == [[1, 2, 0, -1], [-1] * 4, [0, 2, 4, 3], [-1] * 4]
    assert w[1].tolist() == [0.0] * 4 and w[3].tolist() == [0.0] * 4
    assert ob.gate_ref(l, 2, "softmax")[1][2].tolist() == [0.5, 0.5]
    # the bias chooses, the score weighs
    ids, w = ob.gate_ref(l[3:], 1, "sigmoid", torch.tensor([9.0, 0, 0, 0, 0]), renorm=False)
    assert ids.tolist() == [[0]] and float(w) == 0.5


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("off", [None, [0, 2, 2, 5], [1, 4]])
def test_balance_loss_by_loops_and_its_gradient(score, off):
    l = _rand(6, 5, seed=11)
    ids = torch.tensor([[0, 1], [2, 0], [4, 3], [-1, 2], [0, 1], [1, 5]], dtype=torch.int32)
    loss, counts, dl, _ = ob.balance_loss_ref(l, ids, 0.3, score, off)
    o = [0, 6] if off is None else off
    B = len(o) - 1

    def by_loops(ll):
        total = 0.0
        for b in range(B):
            n = o[b + 1] - o[b]
            for e in range(5):
                c = sum(1 for t in range(o[b], o[b + 1]) for j in range(2) if int(ids[t, j]) == e)
                assert c == int(counts[b, e])
                for t in range(o[b], o[b + 1]):
                    row = ll[t].tolist()
                    s = [_score_by_loop(row, i, score) for i in range(5)]
                    total += 0.3 / B * (5 * c / (2 * n)) * s[e] / sum(s) / n
        return total
    assert loss == pytest.approx(by_loops(l), rel=1e-12)
    torch.testing.assert_close(dl, _differences(by_loops, l), rtol=1e-6, atol=1e-9)
