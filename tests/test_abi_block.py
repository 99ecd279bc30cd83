"""Host-side argument checks of the operators in front of the FFN, through the C ABI.
Nothing here launches GPU work: every call is refused, or has nothing to do."""

import ctypes

import pytest
import torch

import mxfp4_weights_fp8_amd as moe

P = ctypes.c_void_p(0x1000)       # never dereferenced: every check fails first
ODD = ctypes.c_void_p(0x1008)     # not 16-byte aligned
INF, NAN = float("inf"), float("nan")


def norm(T=4, H=256, eps=1e-6, x=P, res=P, w=P, wt=0, h=P, y=P, q=P, s=P):
    return moe.lib().moe_add_norm(T, H, eps, x, res, w, wt, h, y, q, s, None)


def norm_grad(T=4, H=256, eps=1e-6, dy=P, h=P, w=P, wt=0, dh=P, dx=P, dw=P, ws=P, n=1 << 30):
    return moe.lib().moe_add_norm_grad(T, H, eps, dy, h, w, wt, dh, dx, dw, ws, n, None)


def linear(M=4, N=32, K=128, act=0, type=0, x=P, w=P, b=P, res=P, y=P, z=P, ws=P, n=1 << 40):
    d = moe.LinearDims(M, N, K, act, type)
    return moe.lib().moe_linear(d, x, w, b, res, y, z, ws, n, None)


def linear_grad(M=4, N=32, K=128, act=0, type=0, dy=P, x=P, w=P, z=P, dx=P, dw=P, db=P, ws=P, n=1 << 40):
    d = moe.LinearDims(M, N, K, act, type)
    return moe.lib().moe_linear_grad(d, dy, x, w, z, dx, dw, db, ws, n, None)


def gate(T=4, E=8, K=2, score=0, renorm=1, type=1, scale=1.0, l=P, b=P, nv=P, ids=P, w=P):
    return moe.lib().moe_gate(moe.GateDims(T, E, K, score, renorm, type, scale), l, b, nv, ids, w, None)


def gate_grad(T=4, E=8, K=2, score=0, renorm=1, type=1, scale=1.0, l=P, ids=P, dw=P, add=P, dl=P):
    return moe.lib().moe_gate_grad(moe.GateDims(T, E, K, score, renorm, type, scale), l, ids, dw, add, dl, None)


def balance(T=4, E=8, K=2, B=1, alpha=1.0, score=0, type=1, l=P, ids=P, off=P, loss=P, c=P, dl=P, ws=P, n=1 << 30):
    d = moe.GateDims(T, E, K, score, 0, type, 1.0)
    return moe.lib().moe_balance_loss(d, B, alpha, l, ids, off, loss, c, dl, ws, n, None)


EI, EU, EW = moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED, moe.MOE_EWORKSPACE


@pytest.mark.parametrize("call,kw,code", [
    (norm, dict(T=-1), EI), (norm, dict(H=0), EI), (norm, dict(H=200), EU), (norm, dict(H=16512), EU),
    (norm, dict(T=(1 << 21) + 1), EU), (norm, dict(eps=-1.0), EI), (norm, dict(eps=NAN), EI), (norm, dict(eps=INF), EI),
    (norm, dict(wt=2), EI), (norm, dict(x=None), EI), (norm, dict(w=None), EI), (norm, dict(q=None), EI),
    (norm, dict(s=None), EI), (norm, dict(h=None, y=None, q=None, s=None), EI), (norm, dict(res=ODD), EI),
    (norm, dict(y=ODD), EI), (norm, dict(T=0, x=None), 0),
    (norm_grad, dict(H=100), EU), (norm_grad, dict(dy=None), EI), (norm_grad, dict(h=None), EI),
    (norm_grad, dict(dx=None), EI), (norm_grad, dict(dw=None), EI), (norm_grad, dict(ws=None), EI),
    (norm_grad, dict(dh=ODD), EI), (norm_grad, dict(n=4 * 256 - 1), EW), (norm_grad, dict(T=0, w=None), EI),
    (linear, dict(M=-1), EI), (linear, dict(N=0), EI), (linear, dict(K=0), EI), (linear, dict(K=192), EU),
    (linear, dict(act=5), EI), (linear, dict(act=-1), EI), (linear, dict(type=2), EI), (linear, dict(N=65537), EU),
    (linear, dict(K=65536 + 128), EU), (linear, dict(N=65536, K=32768), EU), (linear, dict(M=(1 << 21) + 1), EU),
    (linear, dict(x=None), EI), (linear, dict(w=None), EI), (linear, dict(y=None), EI), (linear, dict(b=ODD), EI),
    (linear, dict(z=ODD), EI), (linear, dict(M=512, N=384, K=7168, n=16), EW),
    (linear, dict(M=512, N=384, K=7168, ws=None), EI), (linear, dict(M=0, x=None, y=None), 0),
    (linear_grad, dict(K=64), EU), (linear_grad, dict(dy=None), EI), (linear_grad, dict(x=None), EI),
    (linear_grad, dict(w=None), EI), (linear_grad, dict(act=2, z=None), EI), (linear_grad, dict(ws=None), EI),
    (linear_grad, dict(n=64), EW), (linear_grad, dict(dx=ODD), EI), (linear_grad, dict(M=0, dw=None, db=None), 0),
    (gate, dict(T=-1), EI), (gate, dict(E=0), EI), (gate, dict(E=4097), EI), (gate, dict(K=0), EI), (gate, dict(K=9), EI),
    (gate, dict(E=100, K=65), EI), (gate, dict(score=3), EI), (gate, dict(renorm=2), EI), (gate, dict(type=2), EI),
    (gate, dict(scale=INF), EI), (gate, dict(T=(1 << 21) + 1), EU), (gate, dict(l=None), EI), (gate, dict(ids=None), EI),
    (gate, dict(w=None), EI), (gate, dict(nv=ODD), EI), (gate, dict(T=0, l=None), 0),
    (gate_grad, dict(l=None), EI), (gate_grad, dict(ids=None), EI), (gate_grad, dict(dw=None), EI),
    (gate_grad, dict(dl=None), EI), (gate_grad, dict(add=ODD), EI), (gate_grad, dict(T=0), 0),
    (balance, dict(B=0), EI), (balance, dict(alpha=NAN), EI), (balance, dict(B=2, off=None), EI),
    (balance, dict(B=1 << 30), EU), (balance, dict(l=None), EI), (balance, dict(ids=None), EI),
    (balance, dict(loss=None), EI), (balance, dict(c=None), EI), (balance, dict(dl=None), EI),
    (balance, dict(T=513, ws=None), EI), (balance, dict(T=513, n=0), EW), (balance, dict(B=5, n=0), EW), (balance, dict(off=ODD), EI), (balance, dict(K=9), EI),
])
def test_calls_are_refused_on_the_host(call, kw, code):
    assert call(**kw) == code


def test_null_dims():
    L = moe.lib()
    assert L.moe_linear(None, P, P, P, P, P, P, P, 1, None) == EI
    assert L.moe_gate(None, P, P, P, P, P, None) == EI
    assert L.moe_linear_workspace_bytes(None) == 0 and L.moe_balance_loss_workspace_bytes(None, 1) == 0


def test_ffn_quantized_checks():
    L = moe.lib()
    d = moe.make_dims(4, 256, 512, 8, 2)

    def call(d, args, ws=P, n=1 << 40):
        return L.moe_ffn_quantized(ctypes.byref(d), *args, None, P, None, ws, n, None)
    ok = [P] * 11
    assert call(d, ok, n=16) == EW
    assert call(d, ok, ws=None) == EI
    for i in range(11):
        assert call(d, ok[:i] + [None] + ok[i + 1:]) == EI, i
    assert call(d, [ODD] + ok[1:]) == EI
    d512 = moe.make_dims(4, 512, 512, 8, 2)
    assert call(d512, [P, ctypes.c_void_p(0x1002)] + ok[2:]) == EI
    assert call(d512, [P, ctypes.c_void_p(0x1004)] + ok[2:], n=16) == EW     # aligned enough: the next check fails
    assert call(d, [P, ctypes.c_void_p(0x1001)] + ok[2:], n=16) == EW
    for flags in (moe.FLAG_A16, moe.FLAG_NVFP4):
        assert call(moe.make_dims(4, 256, 512, 8, 2, flags=flags), ok) == EI
    assert call(moe.make_dims(4, 200, 512, 8, 2), ok) == EU
    assert call(moe.make_dims(0, 256, 512, 8, 2), [None] * 11, ws=None) == moe.MOE_OK


def test_workspaces():
    L = moe.lib()
    assert L.moe_add_norm_grad_workspace_bytes(5, 256) >= 4 * 256
    assert L.moe_add_norm_grad_workspace_bytes(0, 256) == 0 and L.moe_add_norm_grad_workspace_bytes(5, 100) == 0
    assert L.moe_linear_workspace_bytes(moe.LinearDims(0, 8, 128, 0, 0)) == 0
    M, N, K = 300, 70, 256
    need = L.moe_linear_grad_workspace_bytes(moe.LinearDims(M, N, K, 0, 0))
    assert need > 0 and L.moe_linear_grad_workspace_bytes(moe.LinearDims(0, N, K, 0, 0)) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for f in (lambda: moe.add_norm(x, x[0]), lambda: moe.linear(x, x), lambda: moe.gate(x.float(), 2),
              lambda: moe.add_norm_grad(x, x, x[0]), lambda: moe.linear_grad(x, x, x),
              lambda: moe.gate_grad(x.float(), x, x), lambda: moe.balance_loss(x.float(), x, 1.0),
              lambda: moe.add_norm(x[0], x[0])):
        with pytest.raises(ValueError):
            f()


def test_balance_loss_leaves_one_workgroup_by_work():
    """No workspace: one workgroup does everything. Tokens times experts (times two for
    sqrtsoftplus) decide, not the two of them apart."""
    def need(T, E, B=1, score=0):
        return moe.lib().moe_balance_loss_workspace_bytes(moe.GateDims(T, E, 4, score, 0, 1, 1.0), B)
    assert all(need(*a) == 0 for a in ((512, 64), (256, 256), (64, 512), (7, 384, 1, 2), (64, 64, 4, 1), (64, 384, 4), (0, 512)))
    assert all(need(*a) > 0 for a in ((512, 512), (512, 384, 1, 1), (256, 384, 1, 1), (512, 128, 1, 2), (128, 384, 1, 2), (512, 128, 4, 1)))
