"""GPU tests of the operators in front of the FFN (add_norm, linear, gate, balance_loss
and their gradients) against oracle/block.py in float64, and of a run of them with plan
and ffn_quantized.

Tolerances. u = 2^-24 is half a step of fp32. A rounding to bf16 moves a value by at
most 2^-8 of it, to E4M3 by at most 2^-4 (2^-10 of the scale where it is subnormal). A
sum of n fp32 terms is off by at most n u times the sum of their absolute values; the
kernels add at most `terms` one after another before they go to a tree, so `terms` + a
few stands for n. Functions (exp, erfc, sqrt, division) are taken as 4 u each."""

import math

import numpy as np
import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say, u16
from oracle import block as ob
from oracle.compare import y_metrics
from oracle.formats import dequantize_blocks, scale_exponent
from oracle.moe import ffn_ref, plan_ref
from synth import make_inputs, scaled

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
F64 = torch.float64
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev(gpu):
    moe.lib()
    return gpu


def randn(*shape, seed, scale=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def within(got, want, tol, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    bad = (got - want).abs() - tol
    worst = int(bad.argmax())
    assert float(bad.max()) <= 0, (f"{what}: {int((bad > 0).sum())} values outside; worst got "
                                   f"{float(got.view(-1)[worst])} want {float(want.reshape(-1)[worst])} tolerance "
                                   f"{float(torch.as_tensor(tol).expand_as(want).reshape(-1)[worst])}")


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


# ------------------------------------------------------------------------- add_norm

NORM_TERMS = 8 * 8 + 16     # squares added one after another by a lane, then tree levels


def check_normed(out, x, w, res, eps, what):
    h, y = ob.add_norm_ref(x, w, res, eps)
    rel = (NORM_TERMS / 2 + 16) * U       # half the error of the mean, and a few roundings
    if res is not None:
        within(out.h, h, h.abs() * (BF + 2 * U), what + " h")
    if out.y is not None:
        within(out.y, y, y.abs() * (BF + rel), what + " y")
    if out.x_q is not None:
        codes, scales = out.x_q.cpu().numpy(), out.x_s.cpu().numpy()
        blocks = y.numpy().reshape(-1, 128)
        lo, hi = (scale_exponent(np.abs(blocks).max(1) * f) + 127 for f in (1 - rel, 1 + rel))
        s = scales.reshape(-1).astype(np.int64)
        assert bool(((s == lo) | (s == hi)).all()), what + " scales"
        step = np.exp2(s - 127.0)[:, None]
        v = dequantize_blocks(codes, scales).reshape(-1, 128)
        tol = np.maximum(np.abs(blocks) * 2.0 ** -4, step * 2.0 ** -10) + np.abs(blocks) * 2 * rel
        assert bool((np.abs(v - blocks) <= tol).all()), what + " codes"
        # nearest: never further than the neighbour on either side allows
        assert float(np.sqrt(np.mean((v - blocks) ** 2)) / np.sqrt(np.mean(blocks ** 2))) < 2.0 ** -4


@pytest.mark.parametrize("T,H", [(1, 128), (1, 16384), (7, 7168), (3, 256), (5, 2048), (5, 2176), (2, 4096), (33, 4224),
                                 (2, 8192), (301, 1152), (1, 8320), (2050, 384), (17, 128), (35, 512), (9, 640), (3, 1024),
                                 (49000, 1024)])
@pytest.mark.parametrize("wtype", [BF16, F32])
def test_add_norm(dev, T, H, wtype):
    x, res = randn(T, H, seed=T + H, dtype=BF16), randn(T, H, seed=T + H + 1, scale=3.0, dtype=BF16)
    w = (1 + randn(H, seed=5, scale=0.3)).to(wtype)
    say(f"[add_norm {T}x{H} {wtype}]")
    xd, rd, wd = on(dev, x, res, w)
    out = moe.add_norm(xd, wd, residual=rd, eps=1e-5)
    torch.cuda.synchronize()
    check_normed(out, x, w, res, 1e-5, "with residual")
    alone = moe.add_norm(xd, wd)
    assert alone.h is xd
    check_normed(alone, x, w, None, 1e-6, "without")
    # each output alone gives the same bytes
    only_y, only_q = moe.add_norm(xd, wd, rd, 1e-5, fp8=False), moe.add_norm(xd, wd, rd, 1e-5, bf16=False)
    assert only_y.x_q is None and only_q.y is None
    assert torch.equal(only_y.y, out.y) and torch.equal(only_q.x_q, out.x_q) and torch.equal(only_q.x_s, out.x_s)
    # in place: the residual stream takes h, x takes y
    xi, ri = xd.clone(), rd.clone()
    got = moe.add_norm(xi, wd, ri, 1e-5, out=moe.Normed(ri, xi, None, None))
    assert torch.equal(ri, out.h) and torch.equal(xi, out.y) and torch.equal(got.x_q, out.x_q)


def test_add_norm_rows_of_zeros_infinities_and_large_values(dev):
    H = 256
    x = randn(6, H, seed=3, dtype=BF16)
    x[1] = 0
    x[2, 7] = math.inf
    x[3, 9] = math.nan
    x[4] = x[4] * 1e15
    x[5] = x[5] * 1e-15
    w = torch.ones(H)
    out = moe.add_norm(*on(dev, x, w), eps=1e-6)
    y = out.y.cpu().float()
    assert bool((y[1] == 0).all()) and bool((out.x_q.cpu()[1] == 0).all())
    assert bool(torch.isnan(y[2, 7])) and bool(torch.isnan(y[3]).all())
    keep = [0, 1, 4, 5]      # the other rows are what they are alone
    ref = ob.add_norm_ref(x[keep], w, None, 1e-6)[1]
    within(out.y.cpu()[keep], ref, ref.abs() * (BF + 60 * U) + 1e-38, "rows beside non-finite ones")


@pytest.mark.parametrize("T,H", [(1, 128), (7, 7168), (2, 16384), (1100, 384), (37, 2304), (5, 4096), (19, 128),
                                 (16500, 256), (5003, 1024), (3, 2048), (49000, 1024), (70, 512), (1025, 8320)])
@pytest.mark.parametrize("wtype,with_dh", [(BF16, True), (F32, False)])
def test_add_norm_grad(dev, T, H, wtype, with_dh):
    dy, h = randn(T, H, seed=1, dtype=BF16), randn(T, H, seed=2, scale=2.0, dtype=BF16)
    dh = randn(T, H, seed=3, dtype=BF16) if with_dh else None
    w = (1 + randn(H, seed=4, scale=0.3)).to(wtype)
    dyd, hd, wd, dhd = on(dev, dy, h, w, dh)
    say(f"[add_norm_grad {T}x{H}]")
    dx, dw = moe.add_norm_grad(dyd, hd, wd, eps=1e-5, dh=dhd)
    torch.cuda.synchronize()
    rdx, rdw = ob.add_norm_grad_ref(dy, h, w, 1e-5, dh)
    g, h64 = (dy.to(F64) * w.to(F64)).abs(), h.to(F64).abs()
    r = 1 / ((h64 * h64).mean(1, keepdim=True) + 1e-5).sqrt()
    mag = r * g + r ** 3 * h64 * (g * h64).mean(1, keepdim=True)   # the terms dx adds up
    within(dx, rdx, rdx.abs() * BF + (mag + (0 if dh is None else dh.to(F64).abs())) * (2 * NORM_TERMS + 32) * U, "dx")
    terms = min(T, T // 512 + 1024)      # rows of a workgroup, then the workgroups' parts
    within(dw, rdw, (dy.to(F64).abs() * h64 * r).sum(0) * (terms + NORM_TERMS + 16) * U, "dweight")
    again, dw2 = moe.add_norm_grad(dyd, hd, wd, eps=1e-5, dh=dhd)
    assert torch.equal(dx, again) and torch.equal(dw, dw2)
    inplace = dyd.clone()
    moe.add_norm_grad(inplace, hd, wd, eps=1e-5, dh=dhd, dx=inplace)
    assert torch.equal(inplace, dx)
    if dhd is not None:
        inplace = dhd.clone()
        moe.add_norm_grad(dyd, hd, wd, eps=1e-5, dh=inplace, dx=inplace)
        assert torch.equal(inplace, dx)


def test_add_norm_grad_no_rows(dev):
    e = torch.empty(0, 256, dtype=BF16, device=dev)
    w = torch.ones(256, device=dev)
    dx, dw = moe.add_norm_grad(e, e, w)
    assert dx.shape == (0, 256) and bool((dw == 0).all())
    assert moe.add_norm(e, w).y.shape == (0, 256)


# --------------------------------------------------------------------------- linear

def product_tol(x, w, K):
    """Rounding of an fp32 sum of K exact products: 32 at a time, K / 32 of them in a
    chain (shorter where K is split), twice as much for the matrix unit's own adds."""
    return (x.to(F64).abs() @ w.to(F64).abs().t()) * (K / 32 + 64) * 2 * U


def check_linear(dev, M, N, K, act="none", bias=False, res=False, dtype=BF16, z=False, seed=0):
    x, w = randn(M, K, seed=seed, dtype=BF16), randn(N, K, seed=seed + 1, scale=1 / math.sqrt(K), dtype=BF16)
    b = randn(N, seed=seed + 2) if bias else None
    r = randn(M, N, seed=seed + 3, dtype=dtype) if res else None
    xd, wd, bd, rd = on(dev, x, w, b, r)
    zd = torch.full((M, N), math.nan, device=dev) if z else None
    say(f"[linear {M}x{N}x{K} {act} bias={bias} res={res} {dtype}]")
    y = moe.linear(xd, wd, bias=bd, act=act, residual=rd, dtype=dtype, z=zd)
    torch.cuda.synchronize()
    ry, rz = ob.linear_ref(x, w, b, act, r)
    tz = product_tol(x, w, K) + rz.abs() * 2 * U
    if z:
        within(zd, rz, tz, "z")
    a = ob.act_ref(rz, act).abs()
    ty = 1.2 * tz + (a + ry.abs()) * 16 * U + (ry.abs() * BF if dtype == BF16 else 0)   # slopes are at most 1.13
    within(y, ry, ty, "y")
    assert torch.equal(y, moe.linear(xd, wd, bias=bd, act=act, residual=rd, dtype=dtype)), "not deterministic"
    if res:
        moe.linear(xd, wd, bias=bd, act=act, residual=rd, dtype=dtype, y=rd)
        assert torch.equal(rd, y), "in place"


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 384, 7168), (7, 384, 7168), (16, 17, 256), (17, 16, 384), (33, 100, 1024),
                                   (64, 7, 2048), (3, 4097, 128), (64, 512, 8192), (48, 30, 128),
                                   (8, 769, 640), (5, 2048, 1152), (4, 767, 896), (2, 2049, 256), (40, 384, 7168),
                                   (9, 33, 4096), (1, 770, 8192), (6, 1536, 256), (7, 1537, 1024),
                                   (17, 8192, 7168), (64, 6001, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_few_rows(dev, M, N, K, dtype):
    check_linear(dev, M, N, K, dtype=dtype, bias=N % 2 == 0, res=K < 1024, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(65, 1, 128), (128, 128, 128), (129, 257, 256), (200, 384, 7168), (1000, 384, 1024),
                                   (300, 5, 640), (513, 770, 384), (1025, 192, 128), (4096, 6, 128), (70, 4099, 512),
                                   (2500, 1280, 256), (130, 130, 4096), (97, 333, 8064)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_tiles(dev, M, N, K, dtype):
    check_linear(dev, M, N, K, dtype=dtype, bias=M % 2 == 0, res=N % 2 == 1, seed=M + N)


@pytest.mark.parametrize("M,N,K", [(1000, 8197, 512), (12003, 1000, 512), (16500, 700, 2048),   # 256 x 192, 192 x 256, 256 x 256
                                   (1001, 8200, 128), (8203, 777, 256)])
def test_linear_large_tiles(dev, M, N, K):
    check_linear(dev, M, N, K, act="silu", bias=True, res=True, dtype=F32 if N % 2 else BF16, z=N % 2 == 1, seed=N)


@pytest.mark.parametrize("M,N,K", [(1001, 8200, 128), (8203, 776, 256), (16390, 2504, 384), (70, 8, 128), (257, 120, 384),
                                   (5003, 8008, 128), (4999, 8072, 256), (12003, 1000, 512), (129, 640, 2048)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_without_epilogue(dev, M, N, K, dtype):
    check_linear(dev, M, N, K, dtype=dtype, seed=N)


@pytest.mark.parametrize("M,N", [(9, 33), (150, 72)])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_activations(dev, M, N, act, dtype):
    check_linear(dev, M, N, 256, act=act, bias=True, res=True, dtype=dtype, z=True, seed=M)


def test_linear_large_values_and_nan(dev):
    """Activations far out on both sides; a NaN input row stays in its row."""
    x = torch.zeros(70, 128, dtype=BF16)
    x[:, 0] = torch.linspace(-300, 300, 70).to(BF16)
    w = torch.zeros(3, 128, dtype=BF16)
    w[:, 0] = torch.tensor([1.0, -1.0, 100.0])
    for rows in (70, 20):
        for act in ("relu", "silu", "gelu", "sigmoid"):
            y = moe.linear(*on(dev, x[:rows], w), act=act, dtype=F32)
            ref, _ = ob.linear_ref(x[:rows], w, None, act)
            # a slope below 1.13 times the rounding of an exact z, and 16 u of the value;
            # tails below fp32's normal range go to zero
            within(y, ref, ref.abs() * 300 * U + 1e-37, f"{act} {rows}")
        xn = x[:rows].clone()
        xn[3, 5] = math.nan
        y = moe.linear(*on(dev, xn, w), act="relu", dtype=F32).cpu()
        assert bool(torch.isnan(y[3]).all()) and int(torch.isnan(y).sum()) == 3


def test_linear_no_rows(dev):
    w = randn(4, 128, seed=1, dtype=BF16).to(dev)
    e = torch.empty(0, 128, dtype=BF16, device=dev)
    assert moe.linear(e, w).shape == (0, 4)
    dx, dw, db = moe.linear_grad(torch.empty(0, 4, dtype=BF16, device=dev), e, w)
    assert dx.shape == (0, 128) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("M,N,K,act,dtype", [
    (1, 1, 128, "none", F32), (7, 384, 256, "none", F32), (300, 384, 512, "none", BF16), (129, 70, 384, "silu", BF16),
    (1000, 33, 256, "gelu", F32), (65, 130, 128, "sigmoid", F32), (500, 8, 1024, "relu", BF16),
    (4100, 40, 256, "none", F32), (64, 1000, 128, "none", BF16),
    # every tile shape of both gradients, and runs of column tiles for a short contraction
    (128, 1000, 8192, "none", F32), (128, 12001, 1024, "none", BF16), (2048, 16500, 768, "none", BF16),
    (1000, 500, 8192, "relu", BF16), (12000, 500, 1024, "none", BF16), (16500, 2000, 768, "none", BF16),
    (5003, 300, 2048, "silu", F32), (3001, 120, 4096, "none", BF16),
    (5003, 100, 8064, "none", BF16), (5001, 200, 8064, "relu", BF16), (4997, 300, 8064, "none", BF16)])
def test_linear_grad(dev, M, N, K, act, dtype):
    x, w = randn(M, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=1 / math.sqrt(K), dtype=BF16)
    dy = randn(M, N, seed=3, dtype=dtype)
    z = None if act == "none" else randn(M, N, seed=4, scale=1.5)
    dyd, xd, wd, zd = on(dev, dy, x, w, z)
    say(f"[linear_grad {M}x{N}x{K} {act} {dtype}]")
    dx, dw, db = moe.linear_grad(dyd, xd, wd, act=act, z=zd)
    torch.cuda.synchronize()
    rdx, rdw, rdb, dz = ob.linear_grad_ref(dy, x, w, act, z)
    exact = dtype == BF16 and act == "none"           # dz is bf16 as it is
    op = 0 if exact else BF + 32 * U                  # its rounding to the operand's type, and its slope's
    ax, aw = dz.abs() @ w.to(F64).abs(), dz.abs().t() @ x.to(F64).abs()
    within(dx, rdx, rdx.abs() * BF + ax * (op + (N / 32 + 64) * 2 * U), "dx")
    within(dw, rdw, rdw.abs() * BF + aw * (op + (M / 32 + 64) * 2 * U), "dw")
    within(db, rdb, dz.abs().sum(0) * (32 + 80 + M / 256) * U, "dbias")
    # worst cases aside, roundings to bf16 (here and of the result) average out: about
    # 2^-8 / sqrt(3) each of the result's norm
    for got, want in ((dx, rdx), (dw, rdw)):
        assert float((got.cpu().to(F64) - want).norm() / want.norm()) < 2 * BF / math.sqrt(3)
    # each result alone is the same
    for i in range(3):
        need = tuple(k == i for k in range(3))
        alone = moe.linear_grad(dyd, xd, wd, act=act, z=zd, need=need)
        assert [a is not None for a in alone] == list(need)
        assert torch.equal(alone[i], (dx, dw, db)[i])


def test_linear_grad_is_the_gradient(dev):
    """Directional differences of linear itself (float32 output, products exact)."""
    M, N, K = 40, 24, 128
    x, w, dy = randn(M, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=0.1, dtype=BF16), randn(M, N, seed=3)
    xd, wd, dyd = on(dev, x, w, dy)
    z = torch.empty(M, N, device=dev)
    moe.linear(xd, wd, act="gelu", dtype=F32, z=z)
    dx, dw, _ = moe.linear_grad(dyd, xd, wd, act="gelu", z=z)
    for base, grad, put in ((xd, dx, lambda v: (v, wd)), (wd, dw, lambda v: (xd, v))):
        step = (torch.randn(base.shape, generator=torch.Generator().manual_seed(9)) * 0.02 * float(base.float().std())).to(dev)
        hi, lo = (base.float() + step).to(BF16), (base.float() - step).to(BF16)
        moved = hi.to(F64) - lo.to(F64)               # the step that bf16 kept
        f = [(moe.linear(*put(v), act="gelu", dtype=F32).to(F64) * dyd.to(F64)).sum() for v in (hi, lo)]
        want, got = float(f[0] - f[1]), float((grad.to(F64) * moved).sum())
        # second-order terms cancel in a centred difference; the steps are not quite
        # centred after their rounding: 2 % of the norms' product bounds both
        assert abs(want - got) <= 0.02 * float(grad.to(F64).norm() * moved.norm())


# ----------------------------------------------------------------------------- gate

SCORES = ["softmax", "sigmoid", "sqrtsoftplus"]


def weight_tol(E, spread=24):
    """Relative error of a weight: exponents of up to `spread`, sums of E / 16 terms per
    lane and trees, a few functions."""
    return (2 * spread + E / 16 + 40) * U


def check_gate(dev, logits, K, what, score="softmax", bias=None, renorm=True, scale=1.0, n_valid=None):
    nv = None if n_valid is None else torch.tensor([n_valid], dtype=torch.int32, device=dev)
    ids, w = moe.gate(logits.to(dev), K, score=score, bias=None if bias is None else bias.to(dev), renorm=renorm,
                      scale=scale, n_valid=nv)
    torch.cuda.synchronize()
    rids, rw = ob.gate_ref(logits, K, score, bias, renorm, scale, n_valid)
    same = ids.cpu() == rids
    assert bool(same.all()), f"{what}: rows {(~same).any(1).nonzero().view(-1).tolist()[:5]} pick other experts"
    E = logits.shape[1]
    within(w, rw, rw.abs() * weight_tol(E) + 1e-30, what + " weights")
    return ids, w


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (7, 384, 8), (1, 2, 2), (130, 64, 6), (33, 65, 16), (100, 5, 5), (20, 256, 17),
                                   (65, 500, 10), (9, 1000, 64), (5, 2047, 8), (3, 4096, 64), (21, 130, 1),
                                   (4, 40, 40), (600, 33, 3)])
@pytest.mark.parametrize("score", SCORES)
def test_gate(dev, T, E, K, score):
    l = randn(T, E, seed=T + E, scale=2.0)
    say(f"[gate {T}x{E} top-{K} {score}]")
    check_gate(dev, l, K, "plain", score, renorm=False, scale=1.0)
    check_gate(dev, l, K, "renorm", score, scale=2.5)
    b = randn(E, seed=3, scale=0.1)
    check_gate(dev, l, K, "bias", score, bias=b)
    check_gate(dev, l, K, "bias, padding", score, bias=b, renorm=False, n_valid=T // 2)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E", [64, 37, 700])
def test_gate_bf16_logits_and_ties(dev, score, E):
    """bf16 logits on a coarse grid tie everywhere; with and without a bias the lowest
    index wins, also where the bias itself is tied."""
    l = (randn(50, E, seed=1) * 2).round().div(2).to(BF16)
    for logits in (l, l.float()):
        check_gate(dev, logits, 8, "ties", score)
        check_gate(dev, logits, 8, "ties, equal bias", score, bias=torch.full((E,), 0.25))
        check_gate(dev, logits, 8, "ties, zero bias", score, bias=torch.zeros(E))
    check_gate(dev, torch.zeros(3, E), 8, "all equal", score)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E,K", [(16, 4), (90, 17), (600, 8)])
def test_gate_masks(dev, score, E, K):
    l = randn(12, E, seed=2, scale=3.0)
    inf, low = math.inf, torch.finfo(F32).min
    l[0] = -inf                       # nothing left
    l[1, 1:] = -inf                   # one expert left
    l[2, ::2] = -inf
    l[3, 3] = math.nan
    l[4, 5] = inf
    l[5] = low                        # the type's lowest value is a value
    l[6, : E - 2] = low
    l[7, 2] = l[7, 3] = inf
    l[8] = -inf
    l[8, E - 1] = low
    l[9] = l[9] * 1e30
    b = randn(E, seed=4, scale=0.1)
    for bias in (None, b):
        for renorm in (False, True):
            check_gate(dev, l, K, f"bias={bias is not None} renorm={renorm}", score, bias=bias, renorm=renorm)
    out = b.clone()
    out[0], out[1], out[2] = -inf, math.nan, inf
    ids, _ = moe.gate(l[10:].to(dev), K, score=score, bias=out.to(dev))
    assert bool((ids[:, 0] == 2).all()) and not bool(((ids == 0) | (ids == 1)).any())


def test_gate_near_ties_need_64_bits(dev):
    """Keys that fp32 cannot tell apart: score + bias differing by 1e-9 and less."""
    E, T = 64, 40
    g = torch.Generator().manual_seed(8)
    l = torch.randn(T, E, generator=g) * 0.5
    b = torch.zeros(E)
    l[:, 1::2] = l[:, 0::2] + 1e-7 * torch.randint(-3, 4, (T, E // 2), generator=g).float()
    for score in SCORES:
        check_gate(dev, l, 8, score, score, bias=b)
        check_gate(dev, l, 8, score + " biased", score, bias=torch.full((E,), 5.0))


@pytest.mark.parametrize("n", [-3, 0, 5, 9, 100])
def test_gate_valid_counts(dev, n):
    check_gate(dev, randn(9, 30, seed=1), 4, f"n_valid={n}", "sigmoid", n_valid=n)


def test_gate_large_scale(dev):
    """Rows without any pick have weights of 0 whatever the scale; the others' stay finite."""
    l = randn(5, 20, seed=1)
    l[1] = -math.inf
    l[3, 2:] = -math.inf
    for score in SCORES:
        for renorm in (False, True):
            check_gate(dev, l, 4, f"scale 2^100 {score} renorm={renorm}", score, renorm=renorm, scale=2.0 ** 100)


def check_gate_grad(dev, l, ids, dw, score, renorm, scale, add, what):
    ld, idd, dwd, addd = on(dev, l, ids, dw, add)
    dl = moe.gate_grad(ld, idd, dwd, score=score, renorm=renorm, scale=scale, add=addd)
    torch.cuda.synchronize()
    ref, mag = ob.gate_grad_ref(l, ids, dw, score, renorm, scale, add)
    # A score below fp32's smallest normal number 2^-126 counts as 0. Each term of dl is a
    # score (or a slope, at most a score) times scale (|dw| + a mean of |dw|) / S, and S is
    # at least 1e-20, so leaving such a score out moves dl by at most
    #   2^-126 * scale * 2 max|dw| / 1e-20   (1e-18 or so)
    lost = 2.0 ** -126 * scale * 2 * float(dw.abs().max()) / 1e-20
    within(dl, ref, mag * 3 * weight_tol(l.shape[1]) + lost, what)
    if add is not None:
        moe.gate_grad(ld, idd, dwd, score=score, renorm=renorm, scale=scale, add=addd, d_logits=addd)
        assert torch.equal(addd, dl), "in place"


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (7, 384, 8), (40, 65, 16), (100, 5, 5), (20, 256, 17), (9, 1000, 64), (3, 4096, 64),
                                   (130, 64, 6), (6, 2050, 3)])
@pytest.mark.parametrize("score", SCORES)
def test_gate_grad(dev, T, E, K, score):
    l = randn(T, E, seed=T + E, scale=2.0)
    ids, _ = ob.gate_ref(l, K, score)
    dw, add = randn(T, K, seed=5), randn(T, E, seed=6)
    say(f"[gate_grad {T}x{E} top-{K} {score}]")
    for renorm in (False, True):
        check_gate_grad(dev, l, ids, dw, score, renorm, 2.5, add, f"renorm={renorm} add")
        check_gate_grad(dev, l.to(BF16), ids, dw, score, renorm, 1.0, None, f"renorm={renorm} bf16")


@pytest.mark.parametrize("score", SCORES)
def test_gate_grad_dropped_doubled_and_masked(dev, score):
    l = randn(6, 20, seed=1, scale=2.0)
    l[2, 4] = -math.inf
    l[3] = -math.inf
    l[4, 1] = -90.0
    l[5, 1] = 90.0
    ids = torch.tensor([[0, 1, 2], [5, 5, 7], [4, 3, -1], [1, 2, 3], [1, 20, -7], [1, 2, 2 ** 31 - 1]], dtype=torch.int32)
    dw = randn(6, 3, seed=2)
    for renorm in (False, True):
        check_gate_grad(dev, l, ids, dw, score, renorm, 1.5, None, f"renorm={renorm}")


# --------------------------------------------------------------------- balance loss

def check_balance(dev, l, ids, alpha, score, off, what):
    o = None if off is None else torch.tensor(off, dtype=torch.int32)
    ld, idd, od = on(dev, l, ids, o)
    loss, counts, dl = moe.balance_loss(ld, idd, alpha, score=score, seq_offsets=od)
    torch.cuda.synchronize()
    rl, rc, rd, mag = ob.balance_loss_ref(l, ids, alpha, score, off)
    assert torch.equal(counts.cpu(), rc), what + " counts"
    tol = 2 * weight_tol(l.shape[1])
    assert abs(float(loss) - rl) <= abs(rl) * tol + 1e-30, (what, float(loss), rl)
    within(dl, rd, mag * 3 * tol + 1e-30, what + " gradient")
    again = moe.balance_loss(ld, idd, alpha, score=score, seq_offsets=od)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, dl))), "not deterministic"


@pytest.mark.parametrize("T,E,K", [(1, 2, 1), (7, 384, 8), (300, 64, 6), (1000, 5, 2), (130, 257, 16), (70, 1000, 64), (5, 4096, 8)])
@pytest.mark.parametrize("score", SCORES)
def test_balance_loss(dev, T, E, K, score):
    l = randn(T, E, seed=T, scale=1.5) + randn(E, seed=3)
    ids, _ = ob.gate_ref(l, K, score)
    ids[::7, 0] = -1
    ids[::11, K - 1] = E
    say(f"[balance {T}x{E} top-{K} {score}]")
    check_balance(dev, l, ids, 0.3, score, None, "one sequence")
    cut = sorted([0, T // 3, T // 3, T - T // 5])
    check_balance(dev, l, ids, 0.3, score, cut, "sequences, rows behind")
    check_balance(dev, l.to(BF16), ids, 2.0, score, [T // 4, T], "rows in front, bf16")


@pytest.mark.parametrize("score", SCORES)
def test_balance_loss_masks_and_empty(dev, score):
    l = randn(200, 48, seed=1, scale=2.0)
    l[3] = -math.inf
    l[5, 3:] = -math.inf
    l[7, 0] = math.inf
    l[9, 1] = math.nan
    l[11] = torch.finfo(F32).min
    ids, _ = ob.gate_ref(l, 4, score)
    check_balance(dev, l, ids, 1.0, score, None, "masks")
    check_balance(dev, l, ids, 1.0, score, [0, 0, 0, 100, 100, 200, 200], "empty sequences")
    check_balance(dev, l, ids, 1.0, score, [50, 50], "no token in any")
    check_balance(dev, l, ids, 1.0, score, list(range(201)), "one token each")
    check_balance(dev, l, ids, 1.0, score, list(range(0, 201, 2)), "two tokens each")
    check_balance(dev, l, ids, 1.0, score, [7] * 150 + list(range(7, 180)), "more than 256 sequences")
    check_balance(dev, l, torch.full_like(ids, -1), 1.0, score, None, "every pick dropped")


def test_balance_loss_no_tokens(dev):
    for E in (8, 600):
        loss, counts, dl = moe.balance_loss(torch.empty(0, E, device=dev), torch.empty(0, 2, dtype=torch.int32, device=dev), 1.0)
        assert float(loss) == 0 and bool((counts == 0).all()) and dl.shape == (0, E)


def test_balance_loss_unordered_offsets_stay_in_bounds(dev):
    """Documented as unspecified values: the call returns and writes its buffers only."""
    l, ids = randn(100, 16, seed=1), torch.zeros(100, 2, dtype=torch.int32)
    off = torch.tensor([0, 90, 10, 1000, 50, 100], dtype=torch.int32)
    ld, idd, od = on(dev, l, ids, off)
    loss, counts, dl = moe.balance_loss(ld, idd, 1.0, seq_offsets=od)
    torch.cuda.synchronize()
    assert counts.shape == (5, 16) and dl.shape == (100, 16)



# ------------------------------------------------------------ offsets past 32 bits


@pytest.fixture
def room(dev):
    yield
    torch.cuda.empty_cache()


def tail_rows(dev, rows, cols, last, dtype=BF16, fill=0.0):
    """[rows, cols] of `fill` whose last rows are `last`."""
    t = torch.full((rows, cols), fill, dtype=dtype, device=dev)
    t[rows - last.shape[0]:] = last.to(dev)
    return t


def test_add_norm_past_32_bits(dev, room):
    T, H, n = 300007, 7168, 5                     # 2.15e9 elements
    x, res, w = randn(n, H, seed=1, dtype=BF16), randn(n, H, seed=2, dtype=BF16), 1 + randn(H, seed=3, scale=0.2)
    xd, rd, wd = tail_rows(dev, T, H, x, fill=1.0), tail_rows(dev, T, H, res, fill=1.0), w.to(dev)
    say(f"[add_norm {T}x{H}]")
    out = moe.add_norm(xd, wd, residual=rd)
    check_normed(moe.Normed(*(t[-n:] for t in out)), x, w, res, 1e-6, "last rows")
    check_normed(moe.Normed(*(t[:n] for t in out)), torch.ones(n, H, dtype=BF16), w, torch.ones(n, H, dtype=BF16), 1e-6, "first rows")
    say(f"[add_norm_grad {T}x{H}]")
    dy = tail_rows(dev, T, H, x)                  # zeros, so that dweight is the last rows' alone
    dx, dw = moe.add_norm_grad(dy, rd, wd)
    small, dw_small = moe.add_norm_grad(x.to(dev), res.to(dev), wd)
    assert torch.equal(dx[-n:], small) and not bool(dx[:1000].any())
    rdw = ob.add_norm_grad_ref(x, res, w, 1e-6, None)[1]
    h64 = res.to(F64)
    tol = (x.to(F64).abs() * h64.abs() / ((h64 * h64).mean(1, keepdim=True) + 1e-6).sqrt()).sum(0) * (n + NORM_TERMS + 16) * U
    within(dw, rdw, tol, "dweight")
    within(dw_small, rdw, tol, "dweight of the rows alone")


def test_linear_past_32_bits(dev, room):
    n = 70
    # the rows of x, then the rows of y without and with an epilogue
    for M, N, K, bias in ((262149, 16, 8192, False), (1048579, 2056, 128, False), (1048579, 2056, 128, True)):
        x, w = randn(n, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=1 / math.sqrt(K), dtype=BF16)
        b = randn(N, seed=3) if bias else None
        say(f"[linear {M}x{N}x{K} bias={bias}]")
        y = moe.linear(tail_rows(dev, M, K, x), *on(dev, w, b))
        ref, z = ob.linear_ref(x, w, b)
        within(y[-n:], ref, product_tol(x, w, K) + ref.abs() * (BF + 16 * U), "last rows")
        within(y[:n], (torch.zeros(n, N) if b is None else b.expand(n, N)).to(F64), BF * (0 if b is None else b.abs().to(F64)), "first rows")
        del y


def test_linear_grad_past_32_bits(dev, room):
    n = 70
    for M, N, K in ((1048579, 2056, 128), (1048579, 16, 2176)):    # dy and dz; x and dx
        x, w = randn(n, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=1 / math.sqrt(K), dtype=BF16)
        dy = randn(n, N, seed=3, dtype=BF16)
        say(f"[linear_grad {M}x{N}x{K}]")
        dx, dw, db = moe.linear_grad(tail_rows(dev, M, N, dy), tail_rows(dev, M, K, x, fill=1.0), w.to(dev))
        rdx, rdw, rdb, dz = ob.linear_grad_ref(dy, x, w, "none", None)
        ax, aw = dz.abs() @ w.to(F64).abs(), dz.abs().t() @ x.to(F64).abs()
        within(dx[-n:], rdx, rdx.abs() * BF + ax * (N / 32 + 64) * 2 * U, "dx")
        assert not bool(dx[:1000].any())
        within(dw, rdw, rdw.abs() * BF + aw * (n / 32 + 64) * 2 * U, "dw")
        within(db, rdb, dz.abs().sum(0) * (n + 64) * U, "dbias")
        del dx, dw, db


def test_router_past_32_bits(dev, room):
    T, E, K, n = 1048579, 2056, 8, 40
    l, dw = randn(n, E, seed=1, scale=2.0), randn(n, K, seed=2)
    ld = tail_rows(dev, T, E, l, dtype=F32)
    say(f"[gate {T}x{E}]")
    ids, w = moe.gate(ld, K)
    rids, rw = ob.gate_ref(l, K, "softmax")
    assert torch.equal(ids[-n:].cpu(), rids)
    within(w[-n:], rw, rw * weight_tol(E), "weights")
    assert bool((ids[:n] == torch.arange(K, device=dev)).all())    # equal logits: the lowest indices
    say(f"[balance_loss {T}x{E}]")
    off = torch.tensor([0, T - n, T], dtype=torch.int32, device=dev)
    loss, counts, dl = moe.balance_loss(ld, ids, 1.0, seq_offsets=off)
    _, rc, rd, mag = ob.balance_loss_ref(l, rids, 0.5, "softmax", None)
    assert torch.equal(counts[1:].cpu(), rc) and int(counts[0, 0]) == T - n
    tol = 6 * weight_tol(E)
    within(dl[-n:], rd, mag * tol + 1e-30, "balance gradient")
    say(f"[gate_grad {T}x{E}]")
    add = dl[-n:].cpu()
    moe.gate_grad(ld, ids, tail_rows(dev, T, K, dw, dtype=F32), add=dl, d_logits=dl)
    rg, mag = ob.gate_grad_ref(l, rids, dw, "softmax", True, 1.0, add)
    within(dl[-n:], rg, mag * 3 * weight_tol(E) + 1e-17, "gradient")

# --------------------------------------------------------- together, graphs, streams

def _block(dev, T, H=512, I=256, E=16, K=4, Is=0, seed=40):
    inp = make_inputs(scaled("tiny", T=T, H=H, I=I, E=E, K=K, Is=Is, seed=seed, weight_seed=seed, name="block")).to(dev)
    extra = {"res": randn(T, H, seed=seed, scale=2.0, dtype=BF16).to(dev),
             "norm": (1 + randn(H, seed=seed + 1, scale=0.2)).to(dev),
             "router": randn(E, H, seed=seed + 2, scale=1 / math.sqrt(H), dtype=BF16).to(dev),
             "bias": randn(E, seed=seed + 3, scale=0.1).to(dev)}
    return inp, extra


def _serve(inp, ex, W, pbuf=None, ws=None, y=None, x=None, res=None):
    w = inp.wl
    n = moe.add_norm(inp.x if x is None else x, ex["norm"], residual=ex["res"] if res is None else res)
    logits = moe.linear(n.y, ex["router"], dtype=F32)
    ids, tw = moe.gate(logits, w.K, score="sigmoid", bias=ex["bias"], scale=1.5)
    p = moe.plan(ids, w.E, w.H, w.I, Is=w.Is if inp.shared else 0, out=pbuf)
    out = moe.ffn_quantized(n.x_q, n.x_s, tw, p, W, shared=inp.shared, ws=ws, y=y)
    return n, logits, ids, tw, p, out


@pytest.mark.parametrize("T,Is", [(7, 0), (300, 128)])
def test_block_from_residual_to_experts(dev, T, Is):
    """add_norm -> router -> gate -> plan -> ffn_quantized, each stage against the oracle
    on what the stage before gave."""
    inp, ex = _block(dev, T, Is=Is)
    w = inp.wl
    n, logits, ids, tw, p, y = _serve(inp, ex, moe.pack_weights(inp.weights))
    torch.cuda.synchronize()
    cpu = {k: v.cpu() for k, v in ex.items()}
    check_normed(n, inp.x.cpu(), cpu["norm"], cpu["res"], 1e-6, "norm")
    ny = n.y.cpu()
    within(logits, ob.linear_ref(ny, cpu["router"])[0], product_tol(ny, cpu["router"], w.H), "logits")
    rids, rw = ob.gate_ref(logits.cpu(), w.K, "sigmoid", cpu["bias"], True, 1.5)
    assert torch.equal(ids.cpu(), rids)
    within(tw, rw, rw * weight_tol(w.E), "weights")
    ref = plan_ref(rids.numpy(), w.E)
    assert np.array_equal(p.sorted_pairs.cpu().numpy(), ref["sorted_pairs"])
    # the codes' values are exact in bf16 and quantize to themselves
    xhat = torch.from_numpy(dequantize_blocks(n.x_q.cpu().numpy(), n.x_s.cpu().numpy())).to(BF16)
    r = ffn_ref(xhat, rids, tw.cpu(), **inp.weights, shared=inp.shared)
    m = y_metrics(u16(y), r["y"])
    say(f"[block T={T} Is={Is}] {m}")
    assert m["finite"] and m["max_rel"] <= 2e-2 and m["mean_rel"] <= 2e-3, m


def test_padded_batch(dev):
    """Rows behind the last token (n_valid): no picks, no part in the plan or the balance
    loss, y zero; the others are what they are without padding."""
    T, n = 40, 27
    inp, ex = _block(dev, T)
    w = inp.wl
    W = moe.pack_weights(inp.weights)
    nv = torch.tensor([n], dtype=torch.int32, device=dev)
    off = torch.tensor([0, n], dtype=torch.int32, device=dev)

    def run(rows, n_valid, seq):
        x = inp.x[:rows].contiguous()
        normed = moe.add_norm(x, ex["norm"], residual=ex["res"][:rows].contiguous())
        logits = moe.linear(normed.y, ex["router"], dtype=F32)
        ids, tw = moe.gate(logits, w.K, score="sigmoid", bias=ex["bias"], n_valid=n_valid)
        p = moe.plan(ids, w.E, w.H, w.I)
        y = moe.ffn_quantized(normed.x_q, normed.x_s, tw, p, W)
        return ids, tw, p, y, moe.balance_loss(logits, ids, 0.1, score="sigmoid", seq_offsets=seq)
    ids, tw, p, y, bal = run(T, nv, off)
    ids1, tw1, p1, y1, bal1 = run(n, None, None)
    torch.cuda.synchronize()
    assert bool((ids[n:] == -1).all()) and bool((tw[n:] == 0).all()) and int(p.status) == (T - n) * w.K
    assert bool((y[n:] == 0).all()) and bool((bal[2][n:] == 0).all())
    assert torch.equal(ids[:n], ids1) and torch.equal(tw[:n], tw1)
    assert torch.equal(y[:n].view(torch.int16), y1.view(torch.int16))
    assert torch.equal(bal[1], bal1[1]) and torch.equal(bal[0], bal1[0]) and torch.equal(bal[2][:n], bal1[2])


@pytest.mark.parametrize("T,Is,flags", [(7, 0, 0), (7, 128, 0), (300, 128, 0), (7, 0, moe.FLAG_DECODE_CHAIN),
                                        (7, 128, moe.FLAG_DECODE_CHAIN), (0, 0, 0)])
def test_ffn_quantized_equals_ffn(dev, T, Is, flags):
    """On moe_quant_act's codes, bit for bit; the workspace starts as NaN bytes."""
    inp, _ = _block(dev, T, Is=Is)
    w = inp.wl
    p = moe.plan(inp.topk_ids, w.E, w.H, w.I, Is=Is, flags=flags)
    W = moe.pack_weights(inp.weights)
    want = moe.ffn(inp.x, inp.topk_weights, p, W, shared=inp.shared)
    x_q, x_s = moe.quant_act(inp.x)
    ws = torch.full((moe.ffn_workspace_bytes(p.dims),), 0xFF, dtype=torch.uint8, device=dev)
    got = moe.ffn_quantized(x_q, x_s, inp.topk_weights, p, W, shared=inp.shared, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T", [7, 300])
@pytest.mark.parametrize("H", [384, 512])
def test_ffn_quantized_on_rows_of_larger_tensors(dev, T, H):
    """Codes and scales that start at a later row: scales at odd addresses where a row has
    three of them."""
    inp, _ = _block(dev, T, H=H)
    w = inp.wl
    W = moe.pack_weights(inp.weights)
    p = moe.plan(inp.topk_ids, w.E, w.H, w.I)
    want = moe.ffn(inp.x, inp.topk_weights, p, W)
    x = torch.cat([inp.x[:1], inp.x])
    x_q, x_s = moe.quant_act(x)
    got = moe.ffn_quantized(x_q[1:], x_s[1:], inp.topk_weights, p, W)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,Is", [(7, 0), (300, 128)])
def test_block_graph_replay(dev, T, Is):
    """The whole block captured into a graph; every replay on new inputs equals an eager
    run, with eager work and synchronizations in between."""
    inp, ex = _block(dev, T, Is=Is)
    W = moe.pack_weights(inp.weights)
    x, res = inp.x.clone(), ex["res"].clone()
    for _ in range(2):
        _serve(inp, ex, W, x=x, res=res)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n, logits, ids, tw, p, y = _serve(inp, ex, W, x=x, res=res)
    for rep in range(3):
        x.copy_(randn(*x.shape, seed=100 + rep, dtype=BF16))
        res.copy_(randn(*x.shape, seed=200 + rep, scale=2.0, dtype=BF16))
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in (n.h, n.y, n.x_q, n.x_s, logits, ids, tw, y)]
        e = _serve(inp, ex, W, x=x, res=res)
        torch.cuda.synchronize()
        for a, b in zip(kept, (e[0].h, e[0].y, e[0].x_q, e[0].x_s, e[1], e[2], e[3], e[5])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep
        say(f"[block graph T={T}] replay {rep} equal to eager")


def _tune(t):
    """A router's tuning step: balance loss, gate, router product and norm, backwards."""
    n = moe.add_norm(t["x"], t["norm"], residual=t["res"], fp8=False)
    logits = moe.linear(n.y, t["router"], dtype=F32)
    ids, tw = moe.gate(logits, 4)
    loss, counts, dl = moe.balance_loss(logits, ids, 0.01, seq_offsets=t["off"])
    dl = moe.gate_grad(logits, ids, t["dtw"], add=dl, d_logits=dl)
    dy, drouter, _ = moe.linear_grad(dl, n.y, t["router"], need=(True, True, False))
    dx, dnorm = moe.add_norm_grad(dy, n.h, t["norm"], dh=t["dh"])
    return loss, counts, dl, drouter, dx, dnorm


def test_router_tuning_step_and_graph(dev):
    T, H, E = 260, 256, 24
    t = {"x": randn(T, H, seed=1, dtype=BF16), "res": randn(T, H, seed=2, scale=2.0, dtype=BF16),
         "norm": 1 + randn(H, seed=3, scale=0.2), "router": randn(E, H, seed=4, scale=0.1, dtype=BF16),
         "dtw": randn(T, 4, seed=5), "dh": randn(T, H, seed=6, dtype=BF16),
         "off": torch.tensor([0, 100, 100, 250], dtype=torch.int32)}
    d = {k: v.to(dev) for k, v in t.items()}
    loss, counts, dl, drouter, dx, dnorm = _tune(d)
    torch.cuda.synchronize()
    # the oracle's step in float64 from start to end; bf16 roundings of y, dz and dy
    # stand between (each 2^-8, of terms that add up like noise: 4 of them bound the norm)
    h, y = ob.add_norm_ref(t["x"], t["norm"], t["res"])
    yb = moe.add_norm(d["x"], d["norm"], residual=d["res"], fp8=False).y.cpu()
    logits = ob.linear_ref(yb, t["router"])[0]
    ids, _ = ob.gate_ref(logits, 4)
    rl, rc, rbal, _ = ob.balance_loss_ref(logits, ids, 0.01, "softmax", [0, 100, 100, 250])
    rdl, _ = ob.gate_grad_ref(logits, ids, t["dtw"], add=rbal)
    rdy, rdr, _, _ = ob.linear_grad_ref(rdl, y, t["router"])
    rdx, rdn = ob.add_norm_grad_ref(rdy, h, t["norm"], dh=t["dh"])
    assert torch.equal(counts.cpu(), rc)
    assert abs(float(loss) - rl) <= 1e-5 * abs(rl)
    for got, want, name in ((dl, rdl, "dlogits"), (drouter, rdr, "drouter"), (dx, rdx, "dx"), (dnorm, rdn, "dnorm")):
        off = float((got.cpu().to(F64) - want).norm() / want.norm())
        say(f"[tuning step] {name} {off:.2e}")
        assert off < 4 * BF, name
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _tune(d)
    for rep in range(3):
        d["x"].copy_(randn(T, H, seed=300 + rep, dtype=BF16))
        d["off"].copy_(torch.tensor([0, 50 + rep, 120, 200 + rep], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in out]
        eager = _tune(d)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager)), rep


def test_two_streams_match_sequential(dev):
    blocks = [(_block(dev, T, seed=s), s) for T, s in ((300, 50), (9, 51))]
    packs = [moe.pack_weights(b[0].weights) for b, _ in blocks]
    want = [_serve(*b, W)[5].clone() for (b, _), W in zip(blocks, packs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for (b, _), W, s in zip(blocks, packs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(_serve(*b, W)[5])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_binding_refuses_wrong_arguments(dev):
    x, w = torch.zeros(4, 256, dtype=BF16, device=dev), torch.zeros(8, 256, dtype=BF16, device=dev)
    l, ids = torch.zeros(4, 8, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    bad = [lambda: moe.add_norm(x, w), lambda: moe.add_norm(x, w[0].half()), lambda: moe.add_norm(x, w[0], residual=x[:2]),
           lambda: moe.add_norm(x.float(), w[0]), lambda: moe.add_norm(x.t(), w[0]), lambda: moe.add_norm(x, w[0].cpu()),
           lambda: moe.linear(x, w[:, :128]), lambda: moe.linear(x, w, act="tanh"), lambda: moe.linear(x, w, dtype=torch.half),
           lambda: moe.linear(x, w, bias=w[:, 0]), lambda: moe.linear(x, w, residual=l),
           lambda: moe.linear_grad(l.double(), x, w), lambda: moe.gate(l, 2, score="tanh"),
           lambda: moe.gate(l.half(), 2), lambda: moe.gate(l, 2, bias=l[0, :4]), lambda: moe.gate(l, 2, n_valid=ids[0]),
           lambda: moe.gate_grad(l, ids, l), lambda: moe.gate_grad(l, ids.long(), l[:, :2].contiguous()),
           lambda: moe.balance_loss(l, ids, 1.0, seq_offsets=ids), lambda: moe.balance_loss(l, ids[:2], 1.0)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.gate(l, 9), lambda: moe.add_norm(x[:, :128].contiguous(), w[0, :128], eps=-1.0),
              lambda: moe.balance_loss(l, ids, float("nan")),
              lambda: moe.balance_loss(l, ids, 1.0, seq_offsets=ids[0, :1].contiguous())):
        with pytest.raises(moe.MoEError):
            f()
