"""GPU tests of the operators that train the experts (rows by expert and back, the
experts' products, the gated activation with its input in 8 bits, and the gradients)
against oracle/train.py in float64, and of a run of them from the norm to the norm's
gradient.

Tolerances. U = 2^-24 is half a step of fp32, BF = 2^-8 of bf16. A sum of n fp32 terms is
off by at most n U times the sum of their absolute values; the matrix unit adds 32
products at a time, n / 32 of them in a chain and a few joins behind it (twice as much
for its own adds). Functions (exp, erfc, division) are taken as 4 U each; an argument's
rounding moves exp(-g) by |g| U and erfc's tail by g^2 U of it."""

import math

import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say
from oracle import block as ob
from oracle import train as ot

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8
F64, BF16, F32, U8 = torch.float64, torch.bfloat16, torch.float32, torch.uint8
ACTS = ["none", "relu", "silu", "gelu", "sigmoid"]
MARK = 7.0       # what buffers hold before a call


@pytest.fixture(scope="module")
def dev(gpu):
    moe.lib()
    return gpu


def randn(*shape, seed, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def within(got, want, tol, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    bad = (got - want).abs() - tol
    if bad.numel():
        worst = int(bad.argmax())
        assert float(bad.max()) <= 0, (f"{what}: {int((bad > 0).sum())} values outside; worst at {worst} got "
                                       f"{float(got.reshape(-1)[worst])} want {float(want.reshape(-1)[worst])}")


def on(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def routed(dev, T, K, E, seed, drop=0.2, H=128):
    """(plan, pair_rows and offsets on the host) of random picks, some of no expert."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < drop] = -1
    p = moe.plan(ids.to(dev), E, H, 128)
    return p, p.pair_rows.cpu(), p.expert_offsets.cpu()


def sized(dev, sizes, K=1, behind=0):
    """A plan whose experts have these numbers of rows, `behind` picks dropped."""
    ids = torch.repeat_interleave(torch.arange(len(sizes), dtype=torch.int32), torch.tensor(sizes))
    ids = torch.cat([ids, torch.full((behind,), -1, dtype=torch.int32)])
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(3))]
    assert ids.numel() % K == 0
    p = moe.plan(ids.view(-1, K).to(dev), len(sizes), 128, 128)
    return p, p.expert_offsets.cpu()


def marked(dev, *shape, dtype=BF16):
    return torch.full(shape, MARK, dtype=dtype, device=dev)


# ------------------------------------------------------------------- rows and back

ROWS = [(1, 1, 8, 1), (1, 8, 7168, 4), (7, 8, 7168, 384), (3, 64, 128, 70), (33, 5, 1000, 9), (2, 2, 16384, 3),
        (300, 4, 264, 8), (5, 9, 520, 4096), (129, 3, 1032, 2), (4100, 2, 136, 17), (61, 7, 512, 12)]


@pytest.mark.parametrize("T,K,H,E", ROWS)
def test_sort_rows(dev, T, K, H, E):
    p, pr, _ = routed(dev, T, K, E, seed=T + H)
    x = randn(T, H, seed=1, dtype=BF16)
    say(f"[sort_rows {T}x{K} of {E}, {H}]")
    out = marked(dev, T * K, H)
    got = moe.sort_rows(x.to(dev), p, rows=out)
    assert got is out
    want = torch.full((T * K, H), MARK, dtype=BF16)
    for r, v in ot.sort_rows_ref(x, pr, T, K).items():
        want[r] = v.to(BF16)
    assert torch.equal(out.cpu(), want)
    if H % 128 == 0:      # from codes: the values they stand for, every one a bf16 value
        q, s = moe.quant_act(x.to(dev))
        val = ot.restored_ref(q.cpu(), s.cpu())
        assert torch.equal(val.to(BF16).to(F64), val)
        moe.sort_rows(q, p, scales=s, rows=out)
        for r, v in ot.sort_rows_ref(val, pr, T, K).items():
            want[r] = v.to(BF16)
        assert torch.equal(out.cpu(), want)
        assert torch.equal(moe.restore_act(q, s).cpu(), val.to(BF16))


def test_every_code_and_scale_is_restored(dev):
    """All 256 codes under every scale that a finite bf16 block takes (bytes 0 .. 247)."""
    q = torch.arange(256, dtype=torch.int32).to(U8).repeat(248, 1)
    s = torch.arange(248, dtype=torch.int32).to(U8)[:, None].repeat(1, 2)
    got = moe.restore_act(*on(dev, q, s)).cpu()
    want = ot.restored_ref(q, s)
    assert torch.equal(torch.isnan(got.to(F64)), torch.isnan(want))
    # codes of 256 and more times 2^120 are 2^128 and more, and bf16 ends at (2 - 2^-7) 2^127: infinite
    past = want.abs() >= 2.0 ** 128
    assert torch.equal(got.to(F64)[past], torch.copysign(torch.full_like(want, math.inf), want)[past])
    ok = ~torch.isnan(want) & ~past
    # values below bf16's smallest step (2^-133) are rounded, to nearest
    assert bool(((got.to(F64) - want).abs()[ok] <= 2.0 ** -134).all())
    big = ok & (want.abs() >= 2.0 ** -126)
    assert torch.equal(got.to(F64)[big], want[big])


@pytest.mark.parametrize("T,K,H,E", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_return_rows_and_its_gradient(dev, T, K, H, E, dtype):
    p, pr, off = routed(dev, T, K, E, seed=T + H)
    live = int(off[-1])
    rows, w, add = randn(T * K, H, seed=1, dtype=BF16), randn(T, K, seed=2), randn(T, H, seed=3, dtype=dtype)
    rows[live:] = math.nan          # nobody's rows
    rd, wd, ad = on(dev, rows, w, add)
    say(f"[return_rows {T}x{K} of {E}, {H} {dtype}]")
    clean = torch.where(torch.isnan(rows), torch.zeros_like(rows), rows)
    out = BF if dtype == BF16 else U
    for weights, more in ((None, None), (wd, ad), (wd, None)):
        y = moe.return_rows(rd, p, weights=weights, add=more, dtype=dtype)
        ry, mag = ot.return_rows_ref(clean, pr, T, K, None if weights is None else w, None if more is None else add)
        within(y, ry, ry.abs() * out + mag * (K + 2) * U, "y")
    again = moe.return_rows(rd, p, weights=wd, add=ad, dtype=dtype, y=ad)
    assert again is ad and torch.equal(ad, moe.return_rows(rd, p, weights=wd, add=add.to(dev), dtype=dtype)), "in place"
    dy = randn(T, H, seed=4, dtype=dtype)
    rdr, rdw, mag = ot.return_rows_grad_ref(dy, clean, pr, T, K, w)
    buf = marked(dev, T * K, H)
    d_rows, d_w = moe.return_rows_grad(dy.to(dev), rd, p, wd, d_rows=buf)
    assert d_rows is buf
    want = torch.full((T * K, H), MARK, dtype=F64)
    for r, v in rdr.items():
        want[r] = v
    within(d_rows, want, want.abs() * (BF + 2 * U), "d_rows")
    assert bool((d_rows.cpu()[live:] == MARK).all())
    # a lane of 64 (16 up to 512 columns) adds H / 64 (H / 16) products, then levels of a tree
    within(d_w, rdw, mag * (H / (16 if H <= 512 else 64) + 16) * U, "d_weights")
    assert bool((d_w.cpu()[pr[:T * K].view(T, K) < 0] == 0).all())
    alone, none = moe.return_rows_grad(dy.to(dev), None, p, wd, need=(True, False))
    assert none is None and torch.equal(alone[:live], d_rows[:live])
    none, only = moe.return_rows_grad(dy.to(dev), rd, p, wd, need=(False, True))
    assert none is None and torch.equal(only, d_w)
    moe.return_rows_grad(dy.to(dev), rd, p, wd, d_rows=rd)
    assert torch.equal(rd[:live], d_rows[:live]) and bool(torch.isnan(rd[live:]).all()), "in place"
    plain, _ = moe.return_rows_grad(dy.to(dev), None, p, need=(True, False))   # without weights: dy itself
    if dtype == BF16:
        assert torch.equal(plain[:live], moe.sort_rows(dy.to(dev), p)[:live])


def test_tokens_without_picks_and_no_tokens(dev):
    ids = torch.full((5, 3), -1, dtype=torch.int32, device=dev)
    p = moe.plan(ids, 4, 128, 128)
    rows = torch.full((15, 128), math.nan, dtype=BF16, device=dev)
    assert bool((moe.return_rows(rows, p) == 0).all())
    add = randn(5, 128, seed=1, dtype=BF16).to(dev)
    assert torch.equal(moe.return_rows(rows, p, weights=torch.ones(5, 3, device=dev), add=add), add)
    _, dw = moe.return_rows_grad(add, rows, p)
    assert bool((dw == 0).all())
    p = moe.plan(torch.empty(0, 3, dtype=torch.int32, device=dev), 4, 128, 128)
    e = torch.empty(0, 128, dtype=BF16, device=dev)
    assert moe.sort_rows(e, p).shape == (0, 128) and moe.return_rows(e, p).shape == (0, 128)
    assert [t.shape for t in moe.return_rows_grad(e, e, p)] == [(0, 128), (0, 3)]
    w = randn(4, 256, 128, seed=2, dtype=BF16).to(dev)
    assert moe.expert_linear(e, w, p).shape == (0, 256)
    dx, dw = moe.expert_linear_grad(torch.empty(0, 256, dtype=BF16, device=dev), e, w, p)
    assert dx.shape == (0, 128) and dw.shape == w.shape and bool((dw == 0).all())
    assert moe.glu(torch.empty(0, 256, dtype=BF16, device=dev))[0].shape == (0, 128)
    assert moe.glu_grad(e, torch.empty(0, 256, dtype=BF16, device=dev))[0].shape == (0, 256)


def test_infinities_stay_in_their_rows(dev):
    p, pr, off = routed(dev, 40, 2, 5, seed=1, drop=0.0)
    rows = randn(80, 128, seed=2, dtype=BF16)
    rows[int(pr[6])] = math.inf          # token 3's first pick
    y = moe.return_rows(rows.to(dev), p).cpu()
    assert bool(torch.isinf(y[3]).all()) and bool(torch.isfinite(y[torch.arange(40) != 3]).all())
    x = randn(40, 128, seed=3, dtype=BF16)
    x[3, 5] = math.nan
    w = randn(5, 128, 128, seed=4, dtype=BF16)
    xr = moe.sort_rows(x.to(dev), p)
    for big in (False, True):            # few rows, and tiles
        if big:
            p, off = sized(dev, [90, 0, 300, 5, 20100], behind=1)
            assert in_tiles(20496, 128, 128, 5)
            xr = randn(20496, 128, seed=5, dtype=BF16).to(dev)
            xr[100, 7] = math.nan
        z = moe.expert_linear(xr, w.to(dev), p).cpu()
        nan_rows = torch.isnan(xr.cpu()).any(1)
        live = int(off[-1])
        assert torch.equal(torch.isnan(z[:live]).all(1), nan_rows[:live])
        assert torch.equal(torch.isnan(z[:live]).any(1), nan_rows[:live])
    d = randn(20496, 128, seed=6, dtype=BF16).to(dev)
    _, dw = moe.expert_linear_grad(d, xr, w.to(dev), p)
    hit = torch.isnan(dw).flatten(1).any(1).cpu().tolist()
    assert hit == [False, False, True, False, False]         # row 100 is expert 2's


# --------------------------------------------------------------- the experts' products

def check_products(dev, sizes, N, C, behind=0, dtype=BF16, seed=0, grad=True):
    p, off = sized(dev, sizes, behind=behind)
    P, E, live = sum(sizes) + behind, len(sizes), sum(sizes)
    x, w = randn(P, C, seed=seed, dtype=BF16), randn(E, N, C, seed=seed + 1, scale=1 / math.sqrt(C), dtype=BF16)
    dy = randn(P, N, seed=seed + 2, dtype=BF16)
    x[live:] = math.nan
    dy[live:] = math.nan
    xd, wd, dyd = on(dev, x, w, dy)
    out = BF if dtype == BF16 else U
    say(f"[experts {len(sizes)} of {P} rows, {N}x{C} {dtype}]")
    y = marked(dev, P, N, dtype=dtype)
    assert moe.expert_linear(xd, wd, p, dtype=dtype, y=y) is y
    torch.cuda.synchronize()
    ry, my = ot.expert_linear_ref(x[:live], w, off)
    within(y[:live], ry, ry.abs() * out + my * (C / 32 + 64) * 2 * U, "y")
    assert bool((y[live:] == MARK).all()), "rows behind the last expert's"
    assert torch.equal(y[:live], moe.expert_linear(xd, wd, p, dtype=dtype)[:live]), "not deterministic"
    if not grad:
        return
    dx = marked(dev, P, C)
    got, dw = moe.expert_linear_grad(dyd, xd, wd, p, dtype=dtype, dx=dx)
    torch.cuda.synchronize()
    assert got is dx
    rdx, rdw, mx, mw = ot.expert_linear_grad_ref(dy[:live], x[:live], w, off)
    within(dx[:live], rdx, rdx.abs() * BF + mx * (N / 32 + 64) * 2 * U, "dx")
    assert bool((dx[live:] == MARK).all()), "rows of dx behind the last expert's"
    within(dw, rdw, rdw.abs() * out + mw * (max(sizes) / 32 + 64) * 2 * U, "dw")
    for need in ((True, False), (False, True)):
        a, b = moe.expert_linear_grad(dyd, xd if need[1] else None, wd if need[0] else None, p, need=need, dtype=dtype)
        assert (a is None) != need[0] and (b is None) != need[1]
        assert b is not None or torch.equal(a[:live], dx[:live])
        assert a is not None or torch.equal(b, dw)


def in_tiles(rows, N, C, E):
    """Whether the forward product runs in tiles (then it has a list in its workspace)."""
    return moe.lib().moe_expert_linear_workspace_bytes(moe.ExpertDims(rows, N, C, E, 0)) > 0


def with_filler(sizes, N, C):
    """These experts and one more, with as many rows as the product needs to run in tiles."""
    n = 0
    while not in_tiles(sum(sizes) + n, N, C, len(sizes) + 1):
        n += 61
    return sizes + [n]


# few rows per expert: one to 64 in a unit, more units, more experts than lanes
@pytest.mark.parametrize("sizes,N,C", [
    ([1], 128, 128), ([0, 3, 0], 128, 256), ([16, 17, 0, 1, 33, 32], 384, 128), ([15, 2, 0, 0, 9], 128, 1152),
    ([64, 0, 0, 0, 0, 1], 256, 384), ([65, 0, 0, 0, 0, 0, 0, 0, 0], 128, 7168), ([0] * 70 + [3, 130] + [0] * 60 + [7], 128, 128),
    ([1] * 200, 128, 384), ([0] * 4000 + [2, 5], 128, 128), ([2] * 65, 256, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_of_few_rows(dev, sizes, N, C, dtype):
    assert not in_tiles(sum(sizes) + 3, N, C, len(sizes))
    check_products(dev, sizes, N, C, behind=3, dtype=dtype, seed=N)


# tiles: sizes around the tiles' 64, 128 and 256 rows; every tile width (256, 192, 128) of
# results and gradients; one step of the contraction and many
@pytest.mark.parametrize("sizes,N,C", [
    ([100], 128, 128), ([64, 65, 127, 128, 129], 256, 128), ([255, 256, 257, 0, 1], 128, 256), ([0, 513, 0, 40], 384, 384),
    ([63, 0, 1025, 2], 640, 256), ([300, 700], 256, 1152), ([17] * 40, 384, 640), ([1, 900, 3], 896, 512),
    ([33, 190, 191, 192, 193], 768, 768), ([20] * 130, 128, 640), ([2100, 5], 256, 2304), ([130] * 20, 1280, 256),
    ([400], 128, 3200), ([300, 90, 0, 513, 33, 700], 2176, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_in_tiles(dev, sizes, N, C, dtype):
    check_products(dev, with_filler(sizes, N, C), N, C, behind=37, dtype=dtype, seed=N + C)


@pytest.mark.parametrize("sizes,N,C", [([5000, 0, 7000, 300, 1200], 512, 1024), ([700] * 24, 768, 256),
                                       ([90] * 384, 256, 384)])
def test_products_of_many_tiles(dev, sizes, N, C):
    assert in_tiles(sum(sizes), N, C, len(sizes))
    check_products(dev, sizes, N, C, seed=N)


# few tiles: the contraction of the product, of dx (over N), of dw (over the rows) in parts
@pytest.mark.parametrize("sizes,N,C,split", [
    ([300], 256, 7168, "y"), ([150, 0, 200, 160, 3], 256, 7168, "y"), ([700], 7168, 128, "dx"), ([90, 300, 0, 257], 4096, 256, "dx"),
    ([3000], 128, 128, "dw"), ([5000, 0, 130, 700], 128, 256, "dw"), ([20000, 1], 256, 128, "dw"), ([64 * 40 + 1], 384, 128, "dw")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_products_in_parts(dev, sizes, N, C, split, dtype):
    P, E = sum(sizes) + 5, len(sizes)
    d = moe.ExpertDims(P, N, C, E, 0)
    if split == "y":
        assert moe.lib().moe_expert_linear_workspace_bytes(d) > 8 * P * N
    else:
        assert moe.lib().moe_expert_linear_grad_workspace_bytes(d) > 8 * (P * C if split == "dx" else E * N * C)
    check_products(dev, sizes, N, C, behind=5, dtype=dtype, seed=N + C)


def test_products_with_most_experts(dev):
    for sizes in ([(7 * i) % 41 for i in range(4096)], [i % 2 for i in range(4096)]):
        check_products(dev, sizes, 128, 128, behind=11)


def test_offsets_past_32_bits(dev):
    """x, y and dx of more than 2^32 bytes, dw and w of more than 2^31 elements' bytes."""
    E, N, C = 3, 128, 16384
    sizes = [70000, 200, 70000]
    p, off = sized(dev, sizes)
    P = sum(sizes)
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(P, C, generator=g, device=dev, dtype=F32).to(BF16)
    assert x.numel() * 2 > 2 ** 32
    w = torch.randn(E, N, C, generator=g, device=dev).mul_(1 / 128).to(BF16)
    dy = torch.randn(P, N, generator=g, device=dev).to(BF16)
    say("[experts, offsets past 32 bits]")
    y = moe.expert_linear(x, w, p)
    dx, dw = moe.expert_linear_grad(dy, x, w, p, dtype=F32)
    torch.cuda.synchronize()
    for r in (0, 69999, 70000, 70199, 70200, P - 130, P - 1):
        e = 0 if r < 70000 else 1 if r < 70200 else 2
        a, b, d = x[r:r + 1].cpu(), w[e:e + 1].cpu(), dy[r:r + 1].cpu()
        one = torch.tensor([0, 1])
        ry, my = ot.expert_linear_ref(a, b, one)
        within(y[r:r + 1], ry, ry.abs() * BF + my * (C / 32 + 64) * 2 * U, f"y of row {r}")
        rdx, _, mx, _ = ot.expert_linear_grad_ref(d, a, b, one)
        within(dx[r:r + 1], rdx, rdx.abs() * BF + mx * (N / 32 + 64) * 2 * U, f"dx of row {r}")
    cols = torch.tensor([0, 1, 8000, C - 1])
    for e, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        a, d = x[lo:hi][:, cols.to(dev)].cpu().to(F64), dy[lo:hi].cpu().to(F64)
        within(dw[e][:, cols.to(dev)], d.t() @ a, (d.abs().t() @ a.abs()) * (len(a) / 32 + 64) * 2 * U, f"dw of expert {e}")
    rows = moe.return_rows_grad(torch.ones(P, C, dtype=BF16, device=dev), None, p, need=(True, False))[0]
    back = moe.return_rows(x, p)
    assert bool((rows[-1] == 1).all()) and torch.equal(back[p.sorted_pairs[P - 1].long()], x[P - 1])


def test_offsets_out_of_order_stay_inside(dev):
    """Offsets that no plan gives: results are unspecified, the buffers' guards are not
    touched and every kernel ends."""
    E, N, C = 5, 256, 128
    for P, k in ((700, 1), (700, -1), (14000, 20)):
        _disorder(dev, E, P, N, C, k)


def _disorder(dev, E, P, N, C, k):
    assert in_tiles(P, N, C, E) == (k == 20)
    p, _ = sized(dev, [P // E] * E)
    x, w, dy = (randn(*s, seed=i, dtype=BF16).to(dev) for i, s in enumerate(((P, C), (E, N, C), (P, N))))
    for bad in ([0, 650, 20, 690, 5, 700], [-9, 100, 2 ** 31 - 1, 300, -2 ** 31, 900], [700, 600, 500, 400, 300, 0]):
        bad = [max(min(v * k, 2 ** 31 - 1), -2 ** 31) for v in bad]
        p.expert_offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        guard = [marked(dev, n + 2 * 4096) for n in (P * N, P * C, E * N * C)]
        y, dx, dw = (t[4096:-4096].view(*s) for t, s in zip(guard, ((P, N), (P, C), (E, N, C))))
        moe.expert_linear(x, w, p, y=y)
        moe.expert_linear_grad(dy, x, w, p, dx=dx, dw=dw)
        torch.cuda.synchronize()
        for t in guard:
            assert bool((t[:4096] == MARK).all()) and bool((t[-4096:] == MARK).all())


def test_product_gradient_is_the_gradient(dev):
    """Directional differences of expert_linear itself (float32 output, products exact)."""
    sizes, N, C = [40, 0, 100, 7], 128, 128
    p, _ = sized(dev, sizes)
    P = sum(sizes)
    x, w, dy = randn(P, C, seed=1, dtype=BF16), randn(4, N, C, seed=2, scale=0.1, dtype=BF16), randn(P, N, seed=3, dtype=BF16)
    xd, wd, dyd = on(dev, x, w, dy)
    dx, dw = moe.expert_linear_grad(dyd, xd, wd, p, dtype=F32)
    for base, grad, put in ((xd, dx, lambda v: (v, wd)), (wd, dw, lambda v: (xd, v))):
        step = (torch.randn(base.shape, generator=torch.Generator().manual_seed(9)) * float(base.float().std())).to(dev)
        hi, lo = (base.float() + step).to(BF16), (base.float() - step).to(BF16)
        moved = hi.to(F64) - lo.to(F64)
        f = [(moe.expert_linear(*put(v), p, dtype=F32).to(F64) * dyd.to(F64)).sum() for v in (hi, lo)]
        want, got = float(f[0] - f[1]), float((grad.to(F64) * moved).sum())
        # bilinear, so differences are exact; the sums' and the gradient's roundings: 2^-8 of the terms
        # (dx is bf16), far below 1 % of the norms' product
        assert abs(want - got) <= 0.01 * float(grad.to(F64).norm() * moved.norm())


# ------------------------------------------------------------------- gated activation

def check_saved(z, q, s, what):
    rq, rs = ot.saved_ref(z)
    assert torch.equal(s.cpu(), rs), what + " scales"
    assert torch.equal(q.cpu(), rq), what + " codes"      # bf16 values scaled by powers of two: exact


def glu_tol(z, out):
    """h = act(g) u: a few functions, their argument's rounding, one rounding."""
    I = z.shape[1] // 2
    return out.abs() * (BF + (32 + 4 * z[:, :I].abs() ** 2) * U) + 1e-37


def check_glu_grad(dz, h, dh, z, act, what):
    rdz, rh = ot.glu_grad_ref(dh, z, act)
    I = rh.shape[1]
    g, u, d = z[:, :I].abs().to(F64), z[:, I:].abs().to(F64), dh.abs().to(F64)
    # the slopes are sums of terms up to 1 + |g| that may cancel
    slope = d * u * (64 + 8 * g * g) * U
    value = d * ob.act_ref(z[:, :I].to(F64), act).abs() * (32 + 4 * g * g) * U
    within(dz, rdz, rdz.abs() * BF + torch.cat([slope, value], 1) + 1e-37, what + " dz")
    if h is not None:
        within(h, rh, glu_tol(z.to(F64), rh), what + " h")


@pytest.mark.parametrize("R,I", [(1, 128), (7, 384), (128, 512), (33, 640), (3, 16384), (1000, 256), (260, 1408)])
@pytest.mark.parametrize("act", ACTS)
def test_glu_and_its_gradient(dev, R, I, act):
    z, dh = randn(R, 2 * I, seed=R, scale=2.0, dtype=BF16), randn(R, I, seed=R + 1, dtype=BF16)
    z[0, :128] = 0                                          # a block of zeros
    zd, dhd = on(dev, z, dh)
    say(f"[glu {R}x{I} {act}]")
    h, q, s = moe.glu(zd, act=act)
    rh = ot.glu_ref(z, act)
    within(h, rh, glu_tol(z.to(F64), rh), "h")
    check_saved(z, q, s, "glu")
    bare, none, _ = moe.glu(zd, act=act, save=False)
    assert none is None and torch.equal(bare, h)
    # from the codes: the gradient at what they stand for
    val = ot.restored_ref(q.cpu(), s.cpu())
    dz, h2 = moe.glu_grad(dhd, q, scales=s, act=act)
    check_glu_grad(dz, h2, dh, val, act, "from codes")
    dz2, none = moe.glu_grad(dhd, q, scales=s, act=act, need_h=False)
    assert none is None and torch.equal(dz2, dz)
    into = dhd.clone()
    dz2, h3 = moe.glu_grad(into, q, scales=s, act=act, out=(None, into))      # h over dh
    assert torch.equal(dz2, dz) and torch.equal(into, h2)
    # from z itself, in place
    dz, h2 = moe.glu_grad(dhd, zd, act=act)
    check_glu_grad(dz, h2, dh, z, act, "from z")
    assert torch.equal(h2, h)
    moe.glu_grad(dhd, zd, act=act, out=(zd, None))
    assert torch.equal(zd, dz)


def test_glu_leaves_rows_of_no_expert(dev):
    p, off = sized(dev, [5, 0, 20], behind=7)
    live, R, I = 25, 32, 256
    z, dh = randn(R, 2 * I, seed=1, dtype=BF16), randn(R, I, seed=2, dtype=BF16)
    z[live:] = math.nan
    zd, dhd = on(dev, z, dh)
    out = (marked(dev, R, I), marked(dev, R, 2 * I, dtype=U8), marked(dev, R, 4, dtype=U8))
    got = moe.glu(zd, p=p, out=out)
    whole = moe.glu(zd[:live].contiguous())
    for a, b, c in zip(got, out, whole):
        assert a is b and torch.equal(a[:live], c) and bool((a[live:] == MARK).all())
    grads = (marked(dev, R, 2 * I), marked(dev, R, I))
    moe.glu_grad(dhd, out[1], scales=out[2], p=p, out=grads)
    for a, c in zip(grads, moe.glu_grad(dhd[:live].contiguous(), whole[1], scales=whole[2])):
        assert torch.equal(a[:live], c) and bool((a[live:] == MARK).all())
    with pytest.raises(ValueError):
        moe.glu(zd[:live].contiguous(), p=p)


def test_glu_past_32_bits(dev):
    """More than 2^31 elements of h, 2^32 of z and dz: the first and the last rows."""
    R, I = 131200, 16384
    z = torch.zeros(R, 2 * I, dtype=BF16, device=dev)
    dh = torch.zeros(R, I, dtype=BF16, device=dev)
    at = [0, 1, 65535, 65536, R - 1]
    assert R * I > 2 ** 31
    some, d = randn(len(at), 2 * I, seed=1, scale=2.0, dtype=BF16), randn(len(at), I, seed=2, dtype=BF16)
    z[at], dh[at] = some.to(dev), d.to(dev)
    h, q, s = moe.glu(z)
    rh = ot.glu_ref(some, "silu")
    within(h[at], rh, glu_tol(some.to(F64), rh), "h")
    check_saved(some, q[at], s[at], "glu")
    assert int((h != 0).any(1).sum()) == len(at)
    dz, h2 = moe.glu_grad(dh, q, scales=s, out=(z, None))
    check_glu_grad(dz[at], h2[at], d, ot.restored_ref(q[at].cpu(), s[at].cpu()), "silu", "gradient")
    assert int((dz != 0).any(1).sum()) == len(at)


def test_binding_refuses_what_the_kernels_cannot_take(dev):
    T, K, E, H, N = 6, 2, 3, 256, 128
    p, _, _ = routed(dev, T, K, E, seed=1, H=H)
    x, rows = randn(T, H, seed=1, dtype=BF16).to(dev), randn(T * K, H, seed=2, dtype=BF16).to(dev)
    w, z = randn(E, N, H, seed=3, dtype=BF16).to(dev), randn(T * K, 2 * N, seed=4, dtype=BF16).to(dev)
    q, s = moe.quant_act(x)
    off = torch.zeros(T * H + 4, dtype=BF16, device=dev)[4:].view(T, H)        # 8 bytes past an aligned address
    wrong = [
        lambda: moe.sort_rows(x.float(), p), lambda: moe.sort_rows(rows, p), lambda: moe.sort_rows(x[:, ::2], p),
        lambda: moe.sort_rows(q, p), lambda: moe.sort_rows(x, p, scales=s), lambda: moe.sort_rows(q, p, scales=s[:, :1]),
        lambda: moe.sort_rows(x, p, rows=rows[:4]), lambda: moe.restore_act(q, s.t()), lambda: moe.restore_act(x, s),
        lambda: moe.return_rows(x, p), lambda: moe.return_rows(rows, p, weights=torch.ones(T, K, dtype=BF16, device=dev)),
        lambda: moe.return_rows(rows, p, add=x.float()), lambda: moe.return_rows(rows, p, dtype=torch.float16),
        lambda: moe.return_rows_grad(x[1:], rows, p), lambda: moe.return_rows_grad(x, x, p),
        lambda: moe.return_rows_grad(x.half(), rows, p),
        lambda: moe.expert_linear(rows, w[:2], p), lambda: moe.expert_linear(x, w, p),
        lambda: moe.expert_linear(rows, w.transpose(1, 2), p), lambda: moe.expert_linear(rows, w.float(), p),
        lambda: moe.expert_linear_grad(z, rows, w, p), lambda: moe.expert_linear_grad(rows[:, :N], rows, w, p),
        lambda: moe.expert_linear_grad(z[:, :N].contiguous(), None, None, p, need=(False, True)),
        lambda: moe.expert_linear_grad(z[:, :N].contiguous(), rows, None, p),
        lambda: moe.glu(z, act="tanh"), lambda: moe.glu(z[:, :255].contiguous()), lambda: moe.glu(x, p=p),
        lambda: moe.glu_grad(rows, z), lambda: moe.glu_grad(z[:, :N].contiguous(), z.to(U8)),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    refused = [
        (lambda: moe.sort_rows(off, p), moe.MOE_EINVAL), (lambda: moe.return_rows_grad(x, None, p), moe.MOE_EINVAL),
        (lambda: moe.return_rows_grad(x, rows, p, need=(False, False)), moe.MOE_EINVAL),
        (lambda: moe.expert_linear_grad(z[:, :N].contiguous(), None, w, p), moe.MOE_EINVAL),
        (lambda: moe.glu(z[:, :N].contiguous()), moe.MOE_EUNSUPPORTED),
        (lambda: moe.expert_linear(rows, w[:, :100].contiguous(), p), moe.MOE_EUNSUPPORTED),
        (lambda: moe.expert_linear_grad(z[:, :N].contiguous(), rows, w, p, ws=torch.empty(16, dtype=U8, device=dev)),
         moe.MOE_EWORKSPACE),
    ]
    for i, (call, code) in enumerate(refused):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.code == code, i


def test_glu_far_out(dev):
    """Gates far out on both sides, blocks of tiny and of huge values."""
    g = torch.cat([torch.linspace(-300, 300, 120), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 104.0, -104.0])])
    z = torch.cat([g, torch.ones(128)])[None].to(BF16).repeat(4, 1)
    z[1] *= 1e-35
    z[2, :128] *= 1e30
    z[3, 128:] *= 1e-3
    dh = torch.ones(4, 128, dtype=BF16)
    zd, dhd = on(dev, z, dh)
    for act in ACTS:
        h, q, s = moe.glu(zd, act=act)
        rh = ot.glu_ref(z, act)
        big = rh.abs() < 3e38
        # tails below the normal range go to zero, and a tail's relative error grows as its
        # argument's rounding does: g^2 U, at most 1 where the tail is still normal (g^2 / 2 < 88)
        tol = rh.abs() * (BF + 1e-4) + 1e-36
        got = h.cpu().to(F64)
        assert bool(((got - rh).abs() <= tol)[big].all()), act
        check_saved(z, q, s, act)
        dz, _ = moe.glu_grad(dhd, zd, act=act)
        rdz, _ = ot.glu_grad_ref(dh, z, act)
        # slopes cancel to a few U of 1 + |g| (of terms that the gate's tail has damped: below 40)
        tol = rdz.abs() * (BF + 1e-4) + 1e-36 + torch.cat([z[:, 128:].abs().to(F64) * 64 * 41 * U, torch.zeros(4, 128)], 1)
        assert bool(((dz.cpu().to(F64) - rdz).abs() <= tol)[:, :].masked_select(rdz.abs() < 3e38).all()), act


# ------------------------------------------------------------------ streams and graphs

def _step(dev, T=96, K=3, E=6, H=256, I=128, seed=1):
    """Everything a training step of the experts calls, on buffers of its own."""
    p, _, _ = routed(dev, T, K, E, seed=seed, H=H)
    x, w, dy = randn(T, H, seed=seed, dtype=BF16).to(dev), torch.rand(T, K, device=dev), randn(T, H, seed=seed + 1, dtype=BF16).to(dev)
    w13 = randn(E, 2 * I, H, seed=seed + 2, scale=1 / math.sqrt(H), dtype=BF16).to(dev)
    w2 = randn(E, H, I, seed=seed + 3, scale=1 / math.sqrt(I), dtype=BF16).to(dev)

    def run():
        q, s = moe.quant_act(x)
        rows = moe.sort_rows(x, p)
        h, zq, zs = moe.glu(moe.expert_linear(rows, w13, p), p=p)
        o = moe.expert_linear(h, w2, p)
        y = moe.return_rows(o, p, weights=w)
        d_o, d_w = moe.return_rows_grad(dy, o, p, w)
        dh, _ = moe.expert_linear_grad(d_o, None, w2, p, need=(True, False))
        dz, h2 = moe.glu_grad(dh, zq, scales=zs, p=p)
        _, dw2 = moe.expert_linear_grad(d_o, h2, None, p, need=(False, True))
        d_rows, dw13 = moe.expert_linear_grad(dz, moe.sort_rows(q, p, scales=s), w13, p)
        dx = moe.return_rows(d_rows, p)
        return y, d_w, dw2, dw13, dx
    return run, (x, w, dy, w13, w2)


@pytest.mark.parametrize("T,E", [(96, 6), (20, 12)])      # tiles, and few rows
def test_graph_replays_equal_eager(dev, T, E):
    run, inputs = _step(dev, T=T, E=E)
    eager = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    other_run, _ = _step(dev, T=T + 7, E=E, seed=9)
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):
        other_out = other_run()
    want_other = [t.clone() for t in other_run()]
    for k in range(4):
        if k == 2:     # new inputs in the same places
            inputs[0].copy_(randn(*inputs[0].shape, seed=50, dtype=BF16))
            eager = [t.clone() for t in run()]
        for t in out:
            t.fill_(math.nan)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b), k
        for a, b in zip(other_out, want_other):
            assert torch.equal(a, b), k


def test_on_another_stream(dev):
    run, _ = _step(dev, T=200, E=5)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    again = run()              # both streams at once
    side.synchronize()
    torch.cuda.synchronize()
    for a, b, c in zip(got, want, again):
        assert torch.equal(a, b) and torch.equal(c, b)


# --------------------------------------------------------------------- the whole layer

@pytest.mark.parametrize("saved", [True, False])
def test_a_layer_and_its_gradients(dev, saved):
    """Norm, router, gate, experts and back, and the gradients of everything down to the
    norm's weight, against float64 autograd of the same layer."""
    T, H, I, E, K = 192, 256, 128, 6, 2
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
    # backward; with `saved` neither y of the norm, nor rows, z or h are kept
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

    leaves = [t.to(F64).requires_grad_() for t in (x, nw, router, w13, w2)]
    lx, lnw, lr, l13, l2 = leaves
    ln = lx / torch.sqrt((lx * lx).mean(1, keepdim=True) + 1e-6) * lnw
    s = torch.sigmoid(ln @ lr.t()).gather(1, ids.cpu().long())
    s = s / (s.sum(1, keepdim=True) + 1e-20)
    ry = torch.zeros(T, H, dtype=F64)
    for t in range(T):
        for j in range(K):
            e = int(ids[t, j])
            v = l13[e] @ ln[t]
            ry[t] = ry[t] + s[t, j] * (l2[e] @ (torch.nn.functional.silu(v[:I]) * v[I:]))
    (ry * dy.to(F64)).sum().backward()

    def off(got, want):
        return float((got.cpu().to(F64) - want).norm() / want.norm())
    # Norms of errors. A rounding to bf16 is at most 2^-8 and 2^-8 / sqrt(3) of the norm on
    # average; a result here is some ten roundings of factors away from its inputs, which
    # add like random numbers: 10^(1/2) 2^-8 = 1.3e-2 bounds them.
    assert off(y, ry.detach()) < 1.3e-2
    # An E4M3 code is off by at most 2^-4 of its value, evenly spread over a step: 2^-4 / sqrt(3) =
    # 3.6e-2 of the norm at most. A gradient takes the code's error of g through act' and act'' and of u
    # directly, and x's in dw: each at most 1.5 times 3.6e-2 (|act'| <= 1.1, g act'' and g act' / act
    # up to 1.3), three of them 9.4e-2.
    most = 9.4e-2 if saved else 1.3e-2
    names = ("dx", "d_norm_weight", "d_router", "dw13", "dw2")
    got = dict(zip(names, (dx, d_nw, d_router, dw13, dw2)))
    for name, leaf in zip(names, leaves):
        e = off(got[name], leaf.grad)
        say(f"[layer, saved={saved}] {name} off by {e:.2e} of its norm")
        assert e < most, name
