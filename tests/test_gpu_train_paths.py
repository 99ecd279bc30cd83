"""GPU tests of the experts' training step in the forms that take a workspace: products in
tiles along their list, and in parts that are joined, in captured graphs, on several
streams at once and in a whole layer; and weights, their gradients and results of more
than 2^31 elements. Tolerances as in test_gpu_train.py."""

import math

import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say
from oracle import train as ot
from test_gpu_train import BF, BF16, F32, F64, U, _step, dev, in_tiles, on, randn, sized, within  # noqa: F401

pytestmark = pytest.mark.gpu


def in_parts(what, rows, N, C, E):
    """Whether the product's y, or its gradient's dx or dw, is computed in parts. The
    gradient's workspace is as large as the larger of dx's and dw's parts: it shows one of
    them where two parts of the other one would not fit."""
    d = moe.ExpertDims(rows, N, C, E, 0)
    if what == "y":
        return moe.lib().moe_expert_linear_workspace_bytes(d) > 8 * rows * N
    parts = {"dx": 8 * rows * C, "dw": 8 * E * N * C}
    return parts.pop(what) < moe.lib().moe_expert_linear_grad_workspace_bytes(d) < parts.popitem()[1]


# tokens, picks, experts, H, I. The first product is 2I x H, the second H x I.
STEPS = [(600, 2, 3, 7168, 128), (3000, 2, 4, 2048, 128)]


def check_paths(T, K, E, H, I):
    P = T * K
    assert in_tiles(P, 2 * I, H, E) and in_tiles(P, H, I, E)
    assert in_parts("y", P, 2 * I, H, E) and not in_parts("y", P, H, I, E)
    if H == 7168:
        assert in_parts("dx", P, H, I, E)        # contracted over H
    else:
        assert in_parts("dw", P, 2 * I, H, E)    # over the rows of few experts


@pytest.mark.parametrize("T,K,E,H,I", STEPS)
def test_graphs_of_tiles_and_parts_replay(dev, T, K, E, H, I):
    check_paths(T, K, E, H, I)
    run, inputs = _step(dev, T=T, K=K, E=E, H=H, I=I)
    eager = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    other_run, _ = _step(dev, T=T + 31, K=K, E=E, H=H, I=I, seed=9)
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        other_out = other_run()
    want_other = [t.clone() for t in other_run()]
    say(f"[graphs {T}x{K} of {E}, {H}, {I}]")
    for k in range(5):
        if k == 2:                               # new inputs in the same places
            inputs[0].copy_(randn(*inputs[0].shape, seed=50, dtype=BF16))
            eager = [t.clone() for t in run()]
        for t in out + other_out:
            t.fill_(math.nan)
        graph.replay()
        other.replay()
        for a, b in zip(run(), eager):           # eager work between the replays
            assert torch.equal(a, b), k
        torch.cuda.synchronize()
        for a, b in zip(out + other_out, eager + want_other):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("T,K,E,H,I", STEPS)
def test_tiles_and_parts_on_streams_at_once(dev, T, K, E, H, I):
    check_paths(T, K, E, H, I)
    steps = [_step(dev, T=T + n, K=K, E=E, H=H, I=I, seed=n + 1)[0] for n in range(3)]
    want = [[t.clone() for t in run()] for run in steps]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in steps]
    say(f"[streams {T}x{K} of {E}, {H}, {I}]")
    got = []
    for _ in range(3):
        for run, side in zip(steps, sides):
            with torch.cuda.stream(side):
                got.append(run())
    for side in sides:
        side.synchronize()
    torch.cuda.synchronize()
    for n, g in enumerate(got):
        for a, b in zip(g, want[n % 3]):
            assert torch.equal(a, b), n


@pytest.mark.parametrize("T,K,E,H,I", STEPS)
@pytest.mark.parametrize("saved", [True, False])
def test_a_layer_in_tiles_and_parts(dev, T, K, E, H, I, saved):
    """Norm, router, gate, experts and back, and all gradients, against float64 autograd."""
    check_paths(T, K, E, H, I)
    x, nw = randn(T, H, seed=1, dtype=BF16), 1 + randn(H, seed=2, scale=0.2)
    router = randn(E, H, seed=3, scale=1.5 / math.sqrt(H), dtype=BF16)
    w13 = randn(E, 2 * I, H, seed=4, scale=1.5 / math.sqrt(H), dtype=BF16)
    w2 = randn(E, H, I, seed=5, scale=1.5 / math.sqrt(I), dtype=BF16)
    dy = randn(T, H, seed=6, dtype=BF16)
    xd, nwd, rd, w13d, w2d, dyd = on(dev, x, nw, router, w13, w2, dy)
    n = moe.add_norm(xd, nwd)
    logits = moe.linear(n.y, rd, dtype=F32)
    ids, wt = moe.gate(logits, K, score="sigmoid")
    p = moe.plan(ids, E, H, I)
    rows = moe.sort_rows(n.y, p)
    z = moe.expert_linear(rows, w13d, p)
    h, zq, zs = moe.glu(z, p=p, save=saved)
    o = moe.expert_linear(h, w2d, p)
    y = moe.return_rows(o, p, weights=wt)
    d_o, d_w = moe.return_rows_grad(dyd, o, p, wt)
    dh, _ = moe.expert_linear_grad(d_o, None, w2d, p, need=(True, False))
    dz, h2 = moe.glu_grad(dh, zq if saved else z, scales=zs, p=p)
    _, dw2 = moe.expert_linear_grad(d_o, h2, None, p, need=(False, True))
    back = moe.sort_rows(n.x_q, p, scales=n.x_s) if saved else rows
    d_rows, dw13 = moe.expert_linear_grad(dz, back, w13d, p)
    d_logits = moe.gate_grad(logits, ids, d_w, score="sigmoid")
    d_n, d_router, _ = moe.linear_grad(d_logits, moe.restore_act(n.x_q, n.x_s) if saved else n.y, rd)
    d_n = moe.return_rows(d_rows, p, add=d_n)
    dx, d_nw = moe.add_norm_grad(d_n, xd, nwd)
    torch.cuda.synchronize()

    lx, lnw, lr, l13, l2 = leaves = [t.to(F64).requires_grad_() for t in (x, nw, router, w13, w2)]
    ln = lx / torch.sqrt((lx * lx).mean(1, keepdim=True) + 1e-6) * lnw
    picks = ids.cpu().long()
    s = torch.sigmoid(ln @ lr.t()).gather(1, picks)
    s = s / (s.sum(1, keepdim=True) + 1e-20)
    ry = torch.zeros(T, H, dtype=F64)
    for e in range(E):
        t, j = (picks == e).nonzero(as_tuple=True)
        v = ln[t] @ l13[e].t()
        ry = ry.index_add(0, t, s[t, j][:, None] * ((torch.nn.functional.silu(v[:, :I]) * v[:, I:]) @ l2[e].t()))
    (ry * dy.to(F64)).sum().backward()

    # bounds of errors' norms: the small layer's in test_gpu_train.py, which no size enters
    assert float((y.cpu().to(F64) - ry.detach()).norm() / ry.detach().norm()) < 1.3e-2
    for name, got, leaf in zip(("dx", "d_norm_weight", "d_router", "dw13", "dw2"), (dx, d_nw, d_router, dw13, dw2), leaves):
        off = float((got.cpu().to(F64) - leaf.grad).norm() / leaf.grad.norm())
        say(f"[layer {T} tokens, saved={saved}] {name} off by {off:.2e} of its norm")
        assert off < (9.4e-2 if saved else 1.3e-2), name


# ------------------------------------------------------------------- past 2^31 elements

@pytest.mark.parametrize("tiles,dtype", [(False, BF16), (True, BF16), (True, F32)])
def test_weights_past_32_bits(dev, tiles, dtype):
    """w and dw of more than 2^31 elements, by the product for few rows and in tiles."""
    E, N, C = 520, 768, 7168
    assert E * N * C > 2 ** 31
    sizes = [60] * E if tiles else [0] * E
    for e, n in ((0, 5), (1, 0), (299, 3), (518, 70), (519, 17)):
        sizes[e] = n
    P, out = sum(sizes), BF if dtype == BF16 else U
    assert in_tiles(P, N, C, E) == tiles
    p, off = sized(dev, sizes)
    g = torch.Generator(device=dev).manual_seed(1)
    w = torch.empty(E, N, C, dtype=BF16, device=dev).normal_(0.0, 1 / math.sqrt(C), generator=g)
    x, dy = randn(P, C, seed=1, dtype=BF16).to(dev), randn(P, N, seed=2, dtype=BF16).to(dev)
    say(f"[experts, {w.numel()} weights, {P} rows]")
    y = moe.expert_linear(x, w, p, dtype=dtype)
    dx, dw = moe.expert_linear_grad(dy, x, w, p, dtype=dtype)
    torch.cuda.synchronize()
    for e in (0, 1, 299, 518, 519):
        lo, hi = int(off[e]), int(off[e + 1])
        one, a, d, b = torch.tensor([0, hi - lo]), x[lo:hi].cpu(), dy[lo:hi].cpu(), w[e:e + 1].cpu()
        ry, my = ot.expert_linear_ref(a, b, one)
        within(y[lo:hi], ry, ry.abs() * out + my * (C / 32 + 64) * 2 * U, f"y of expert {e}")
        rdx, rdw, mx, mw = ot.expert_linear_grad_ref(d, a, b, one)
        within(dx[lo:hi], rdx, rdx.abs() * BF + mx * (N / 32 + 64) * 2 * U, f"dx of expert {e}")
        within(dw[e:e + 1], rdw, rdw.abs() * out + mw * ((hi - lo) / 32 + 64) * 2 * U, f"dw of expert {e}")
    assert int((dw != 0).flatten(1).any(1).sum()) == sum(n > 0 for n in sizes)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_results_past_32_bits(dev, dtype):
    """y and dy of more than 2^31 elements."""
    E, N, C = 3, 16384, 128
    sizes = [70000, 200, 70000]
    P, out = sum(sizes), BF if dtype == BF16 else U
    assert P * N > 2 ** 31
    p, off = sized(dev, sizes)
    g = torch.Generator(device=dev).manual_seed(1)
    w = torch.empty(E, N, C, dtype=BF16, device=dev).normal_(0.0, 1 / math.sqrt(C), generator=g)
    x = torch.empty(P, C, dtype=BF16, device=dev).normal_(generator=g)
    dy = torch.empty(P, N, dtype=BF16, device=dev).normal_(generator=g)
    say(f"[experts, results of {P} x {N}]")
    y = moe.expert_linear(x, w, p, dtype=dtype)
    dx, dw = moe.expert_linear_grad(dy, x, w, p, dtype=dtype)
    torch.cuda.synchronize()
    one = torch.tensor([0, 1])
    for r in (0, 69999, 70000, 70199, 70200, 131072, 131073, P - 1):
        e = 0 if r < 70000 else 1 if r < 70200 else 2
        a, b, d = x[r:r + 1].cpu(), w[e:e + 1].cpu(), dy[r:r + 1].cpu()
        ry, my = ot.expert_linear_ref(a, b, one)
        within(y[r:r + 1], ry, ry.abs() * out + my * (C / 32 + 64) * 2 * U, f"y of row {r}")
        rdx, _, mx, _ = ot.expert_linear_grad_ref(d, a, b, one)
        within(dx[r:r + 1], rdx, rdx.abs() * BF + mx * (N / 32 + 64) * 2 * U, f"dx of row {r}")
    cols = torch.tensor([0, 1, 8000, N - 1])
    for e, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        d, a = dy[lo:hi][:, cols.to(dev)].cpu().to(F64), x[lo:hi].cpu().to(F64)
        want, mag = d.t() @ a, d.abs().t() @ a.abs()
        within(dw[e][cols.to(dev)], want, want.abs() * out + mag * (len(a) / 32 + 64) * 2 * U, f"dw of expert {e}")
