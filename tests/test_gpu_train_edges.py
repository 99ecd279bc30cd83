"""GPU tests of the operators that train the experts at their edges: rows of every number of
picks, gradients of the gated activation where the product of two factors leaves fp32 and
the third brings it back, and where codes stand for more than fp32 holds."""

import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say
from oracle import train as ot
from test_gpu_train import ACTS, BF, BF16, F32, F64, U, check_saved, dev, on, randn, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", list(range(1, 18)) + [63, 64])
@pytest.mark.parametrize("H", [72, 1032])      # waves of several tokens, and of one
def test_return_rows_of_every_number_of_picks(dev, K, H):
    """Tokens with all, some and none of their picks; rows of nobody, and a first row that is
    somebody else's NaN, stay out of them."""
    T, E = 37, 5
    g = torch.Generator().manual_seed(K)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < 0.3] = -1
    ids[4:9], ids[20], ids[36] = -1, 1, 2
    ids[11] = -1
    ids[11, K - 1] = 0
    p = moe.plan(ids.to(dev), E, 128, 128)
    pr, live = p.pair_rows.cpu(), int(p.expert_offsets[-1])
    rows, w = randn(T * K, H, seed=1, dtype=BF16), randn(T, K, seed=2)
    rows[live:] = float("nan")
    first = int((pr[:T * K] == 0).nonzero()) // K         # the token that has row 0
    w[(ids < 0)] = float("nan")                           # weights of dropped picks
    say(f"[return_rows {T}x{K}, {H}]")
    for dtype, out in ((BF16, BF), (F32, U)):
        add = randn(T, H, seed=3, dtype=dtype)
        want, mag = ot.return_rows_ref(rows, pr, T, K, w, add)
        y = moe.return_rows(rows.to(dev), p, weights=w.to(dev), add=add.to(dev), dtype=dtype)
        within(y, want, want.abs() * out + mag * (K + 2) * U, "y")
        bad = rows.clone()
        bad[0] = float("nan")
        y2 = moe.return_rows(bad.to(dev), p, weights=w.to(dev), add=add.to(dev), dtype=dtype)
        rest = torch.arange(T) != first
        assert torch.equal(y2.cpu()[rest], y.cpu()[rest]) and bool(torch.isnan(y2[first]).all())


# Gates whose slope takes 2^134 back into range; each a value that its E4M3 code holds exactly.
TAILS = {"relu": [-1.0, -2.0, -0.0, 0.0], "silu": [-64.0, -72.0, -80.0, -192.0], "gelu": [-8.0, -10.0, -11.0, -12.0],
         "sigmoid": [-64.0, -72.0, -80.0, -6.0]}


@pytest.mark.parametrize("act", list(TAILS))
@pytest.mark.parametrize("R,I", [(3, 128), (700, 12288)])      # stores cached, and past the caches
def test_glu_grad_where_dh_times_u_leaves_fp32(dev, act, R, I):
    """dh u = 2^134 is no fp32 value and dh u act'(g) is one: that, no infinity and no NaN."""
    z, dh = torch.zeros(R, 2 * I), torch.zeros(R, I)
    z[:, :128] = torch.tensor(TAILS[act]).repeat(32)
    z[:, I:I + 128] = 2.0 ** 67 * torch.tensor([1.0, -1.0, 1.25]).repeat(43)[:128]
    dh[:, :128] = 2.0 ** 67 * torch.tensor([1.0, 1.5, -1.0, 1.0, -1.75]).repeat(26)[:128]
    z, dh = z.to(BF16), dh.to(BF16)
    zd, dhd = on(dev, z, dh)
    _, q, s = moe.glu(zd, act=act)
    assert torch.equal(ot.restored_ref(q[:1].cpu(), s[:1].cpu()), z[:1].to(F64))
    want, _ = ot.glu_grad_ref(dh[:1], z[:1], act)
    want = want[:, :I]
    assert bool((want.abs() < 2.0 ** 127).all())
    say(f"[glu_grad far out {R}x{I} {act}]")
    # the slope is off by a few U and its argument's rounding, 2 g^2 U (12^2 for gelu), in all below 2^9 U, and by two
    # steps of fp32 below its normal range, 2^-148, of the 2.2 2^134 that it multiplies
    tol = want.abs() * (BF + 2 ** 9 * U) + 2.0 ** -12
    for what, (dz, _) in (("z", moe.glu_grad(dhd, zd, act=act)), ("codes", moe.glu_grad(dhd, q, scales=s, act=act))):
        assert bool((dz == dz[:1]).all()), what          # the rows are alike, and no NaN
        off = (dz[:1, :I].cpu().to(F64) - want).abs()
        assert bool((off <= tol).all()), what


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R,I", [(2, 128), (700, 12288)])
def test_glu_grad_of_codes_at_the_top(dev, act, R, I):
    """Values from 1.9375 2^127 on are finite in bf16, and their codes stand for 2^128: the
    gradient at 2^128, where it is a number, is that number."""
    top = 2.0 ** 127
    z, dh = torch.zeros(R, 2 * I), torch.zeros(R, I)
    z[0, :128] = top * torch.tensor([1.9921875, -1.9921875, 1.9375, -1.9375, 1.90625, -1.875, 1.0, 0.0]).repeat(16)
    z[0, I:I + 128] = 2.0 ** -100
    z[1, :128] = torch.tensor([-64.0, 0.0, -8.0, -10.0]).repeat(32)
    z[1, I:I + 128] = top * torch.tensor([1.9921875, -1.9375, 1.25, -1.9921875, 1.9375]).repeat(26)[:128]
    dh[:, :128] = 2.0 ** -20 * torch.tensor([1.0, 1.5, -1.0, 1.0, -1.75]).repeat(26)[:128]
    z, dh = z.to(BF16), dh.to(BF16)
    assert bool(torch.isfinite(z).all())
    zd, dhd = on(dev, z, dh)
    _, q, s = moe.glu(zd, act=act)
    check_saved(z[:2], q[:2], s[:2], "top")
    val = ot.restored_ref(q[:2].cpu(), s[:2].cpu())
    assert float(val.max()) == 2.0 ** 128 and float(val.min()) == -2.0 ** 128
    say(f"[glu_grad of codes at the top {R}x{I} {act}]")
    dz, h = moe.glu_grad(dhd, q, scales=s, act=act)
    for got, want in zip((dz, h), ot.glu_grad_ref(dh[:2], val, act)):
        got = got[:2].cpu().to(F64)
        past = want.abs() >= 2.0 ** 128
        assert torch.equal(got[past], torch.copysign(torch.full_like(want, float("inf")), want)[past])
        # as above; 2^128 itself is taken as fp32's largest value, off by U
        assert bool(((got - want).abs() <= want.abs() * (BF + 2 ** 9 * U) + 1e-37)[~past].all())
