"""GPU tests of the operators that train the experts at their edges: gradients of the gated
activation where the product of two factors leaves fp32 and the third brings it back."""

import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say
from oracle import train as ot
from test_gpu_train import BF, BF16, F64, U, dev, on  # noqa: F401

pytestmark = pytest.mark.gpu


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
