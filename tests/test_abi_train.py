"""Host-side argument checks of the operators that train the experts, through the C ABI.
Nothing here launches GPU work: every call is refused, or has nothing to do."""

import ctypes

import pytest
import torch

import mxfp4_weights_fp8_amd as moe

P = ctypes.c_void_p(0x1000)       # never dereferenced: every check fails first
ODD = ctypes.c_void_p(0x1008)     # not 16-byte aligned


def sort(T=4, H=256, K=2, x=P, s=P, pr=P, rows=P):
    return moe.lib().moe_sort_rows(T, H, K, x, s, pr, rows, None)


def restore(T=4, H=256, q=P, s=P, x=P):
    return moe.lib().moe_restore_act(T, H, q, s, x, None)


def back(T=4, H=256, K=2, rows=P, pr=P, w=P, add=P, type=0, y=P):
    return moe.lib().moe_return_rows(T, H, K, rows, pr, w, add, type, y, None)


def back_grad(T=4, H=256, K=2, dy=P, type=0, rows=P, pr=P, w=P, dr=P, dw=P):
    return moe.lib().moe_return_rows_grad(T, H, K, dy, type, rows, pr, w, dr, dw, None)


def product(p=64, N=128, K=128, E=4, type=0, x=P, w=P, off=P, y=P, ws=P, n=1 << 40):
    return moe.lib().moe_expert_linear(moe.ExpertDims(p, N, K, E, type), x, w, off, y, ws, n, None)


def product_grad(p=64, N=128, K=128, E=4, type=0, dy=P, x=P, w=P, off=P, dx=P, dw=P, ws=P, n=1 << 40):
    return moe.lib().moe_expert_linear_grad(moe.ExpertDims(p, N, K, E, type), dy, x, w, off, dx, dw, ws, n, None)


def glu(R=4, I=128, E=2, act=2, z=P, off=P, h=P, q=P, s=P):
    return moe.lib().moe_glu(moe.GluDims(R, I, E, act), z, off, h, q, s, None)


def glu_grad(R=4, I=128, E=2, act=2, dh=P, z=None, q=P, s=P, off=P, dz=P, h=P):
    return moe.lib().moe_glu_grad(moe.GluDims(R, I, E, act), dh, z, q, s, off, dz, h, None)


EI, EU, EW, OK = moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED, moe.MOE_EWORKSPACE, moe.MOE_OK


@pytest.mark.parametrize("call,kw,code", [
    (sort, dict(T=-1), EI), (sort, dict(H=0), EI), (sort, dict(K=0), EI), (sort, dict(K=65), EI), (sort, dict(H=264), EU),
    (sort, dict(H=4, s=None), EU), (sort, dict(H=16392, s=None), EU), (sort, dict(T=(1 << 21) + 1), EU),
    (sort, dict(x=None), EI), (sort, dict(pr=None), EI), (sort, dict(rows=None), EI), (sort, dict(x=ODD), EI),
    (sort, dict(s=ODD), EI), (sort, dict(rows=ODD), EI), (sort, dict(pr=ODD), EI), (sort, dict(T=0, x=None), OK),
    (restore, dict(T=-1), EI), (restore, dict(H=200), EU), (restore, dict(q=None), EI), (restore, dict(s=None), EI),
    (restore, dict(x=None), EI), (restore, dict(q=ODD), EI), (restore, dict(T=0, q=None), OK),
    (back, dict(T=-1), EI), (back, dict(H=-8), EI), (back, dict(H=12), EU), (back, dict(H=16400), EU), (back, dict(K=0), EI),
    (back, dict(type=2), EI), (back, dict(type=2, T=0), EI), (back, dict(rows=None), EI), (back, dict(pr=None), EI),
    (back, dict(y=None), EI), (back, dict(w=ODD), EI), (back, dict(add=ODD), EI), (back, dict(y=ODD), EI),
    (back, dict(T=0, rows=None, y=None), OK),
    (back_grad, dict(T=-1), EI), (back_grad, dict(H=100), EU), (back_grad, dict(K=65), EI), (back_grad, dict(type=-1), EI),
    (back_grad, dict(dy=None), EI), (back_grad, dict(pr=None), EI), (back_grad, dict(rows=None), EI),
    (back_grad, dict(dr=None, dw=None), EI), (back_grad, dict(dy=ODD), EI), (back_grad, dict(dr=ODD), EI),
    (back_grad, dict(dw=ODD), EI), (back_grad, dict(T=0, dy=None), OK),
    (product, dict(p=-1), EI), (product, dict(N=0), EI), (product, dict(K=0), EI), (product, dict(E=0), EI),
    (product, dict(E=4097), EI), (product, dict(type=2), EI), (product, dict(N=192), EU), (product, dict(K=64), EU),
    (product, dict(N=65536 + 128), EU), (product, dict(K=65536 + 128), EU), (product, dict(N=65536, K=32768), EU),
    (product, dict(p=(1 << 27) + 1), EU), (product, dict(x=None), EI), (product, dict(w=None), EI),
    (product, dict(off=None), EI), (product, dict(y=None), EI), (product, dict(x=ODD), EI), (product, dict(off=ODD), EI),
    (product, dict(p=100000, ws=None), EI), (product, dict(p=100000, n=16), EW), (product, dict(p=100000, ws=ODD), EI),
    (product, dict(p=0, x=None, w=None), OK),
    (product_grad, dict(N=100), EU), (product_grad, dict(E=5000), EI), (product_grad, dict(dy=None), EI),
    (product_grad, dict(x=None), EI), (product_grad, dict(w=None), EI), (product_grad, dict(off=None), EI),
    (product_grad, dict(ws=None), EI), (product_grad, dict(n=0), EW), (product_grad, dict(dx=ODD), EI),
    (product_grad, dict(dw=ODD), EI), (product_grad, dict(dx=None, dw=None), OK),
    (product_grad, dict(p=0, dy=None, x=None, w=None, dw=None), OK),
    (glu, dict(R=-1), EI), (glu, dict(I=0), EI), (glu, dict(E=-1), EI), (glu, dict(E=4097), EI), (glu, dict(act=5), EI),
    (glu, dict(act=-1), EI), (glu, dict(I=192), EU), (glu, dict(I=16384 + 128), EU), (glu, dict(z=None), EI),
    (glu, dict(h=None), EI), (glu, dict(q=None), EI), (glu, dict(s=None), EI), (glu, dict(off=None), EI),
    (glu, dict(z=ODD), EI), (glu, dict(q=ODD), EI), (glu, dict(off=ODD), EI), (glu, dict(R=0, z=None), OK),
    (glu_grad, dict(I=64), EU), (glu_grad, dict(act=7), EI), (glu_grad, dict(dh=None), EI), (glu_grad, dict(dz=None), EI),
    (glu_grad, dict(q=None), EI), (glu_grad, dict(s=None), EI), (glu_grad, dict(z=P), EI),
    (glu_grad, dict(q=None, s=None), EI), (glu_grad, dict(off=None), EI), (glu_grad, dict(h=ODD), EI),
    (glu_grad, dict(s=ODD), EI), (glu_grad, dict(R=0, dh=None), OK),
])
def test_calls_are_refused_on_the_host(call, kw, code):
    assert call(**kw) == code


def test_null_dims_and_workspaces():
    L = moe.lib()
    assert L.moe_expert_linear(None, P, P, P, P, P, 1, None) == EI
    assert L.moe_expert_linear_grad(None, P, P, P, P, P, P, P, 1, None) == EI
    assert L.moe_glu(None, P, P, P, P, P, None) == EI and L.moe_glu_grad(None, P, P, P, P, P, P, P, None) == EI
    assert L.moe_expert_linear_workspace_bytes(None) == 0 and L.moe_expert_linear_grad_workspace_bytes(None) == 0
    assert L.moe_expert_linear_workspace_bytes(moe.ExpertDims(0, 128, 128, 4, 0)) == 0
    assert L.moe_expert_linear_workspace_bytes(moe.ExpertDims(100000, 128, 100, 4, 0)) == 0
    assert L.moe_expert_linear_workspace_bytes(moe.ExpertDims(100000, 128, 128, 4, 0)) >= 16 * (100000 // 256 + 4)
    assert L.moe_expert_linear_grad_workspace_bytes(moe.ExpertDims(0, 128, 128, 4, 0)) >= 16


def _plan(T=2, K=2, E=3):
    i32 = torch.int32
    return moe.Plan(moe.make_dims(T, 128, 128, E, K), torch.zeros(E + 1, dtype=i32), torch.zeros(T * K, dtype=i32),
                    torch.zeros(T * K, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1, dtype=torch.uint8))


def test_binding_refuses_cpu_tensors():
    x, p = torch.zeros(2, 128, dtype=torch.bfloat16), _plan()
    rows, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(3, 128, 256, dtype=torch.bfloat16)
    for f in (lambda: moe.sort_rows(x, p), lambda: moe.restore_act(x, x), lambda: moe.return_rows(rows, p),
              lambda: moe.return_rows_grad(x, rows, p), lambda: moe.expert_linear(rows, w, p),
              lambda: moe.expert_linear_grad(rows, rows, w, p), lambda: moe.glu(rows, p=p),
              lambda: moe.glu_grad(x, rows, p=p)):
        with pytest.raises(ValueError):
            f()
