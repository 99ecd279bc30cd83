"""GPU tests of the operators in front of the FFN at their edges: gradients whose dz is no
bf16 value, against the bound that the outputs' own rounding leaves. Tolerances as in
test_gpu_block.py."""

import math
import time

import pytest
import torch

import mxfp4_weights_fp8_amd as moe
from gpu_helpers import say
from oracle import block as ob
from test_gpu_block import BF, BF16, F32, F64, SCORES, U, check_balance, check_gate, check_linear, check_normed, dev, on, randn, room, tail_rows, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- add_norm

@pytest.mark.parametrize("T,H", [(1, 128), (7, 7168), (300, 640)])
def test_add_norm_writes_out_h_without_a_residual(dev, T, H):
    """A buffer given for h receives x, also where h would be x itself, and is checked."""
    x, w = randn(T, H, seed=T, dtype=BF16).to(dev), (1 + randn(H, seed=2, scale=0.2)).to(dev)
    want = moe.add_norm(x, w)
    h = torch.full_like(x, math.nan)
    got = moe.add_norm(x, w, out=moe.Normed(h, None, None, None))
    assert got.h is h and torch.equal(h, x)
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    only = moe.add_norm(x, w, bf16=False, fp8=False, out=moe.Normed(h.fill_(math.nan), None, None, None))
    assert torch.equal(only.h, x) and only[1:] == (None, None, None)
    same = moe.add_norm(x, w, out=moe.Normed(x, None, None, None))
    assert same.h is x and torch.equal(same.y, want.y)
    for bad in (h[:, : H - 1], h.float(), h.cpu()):
        with pytest.raises(ValueError):
            moe.add_norm(x, w, out=moe.Normed(bad, None, None, None))


@pytest.mark.parametrize("T,H", [(127000, 128), (9001, 1920), (2300, 7168), (979, 16384)])
def test_add_norm_past_the_cache(dev, T, H):
    """Tensors that are loaded and stored nontemporally, at every kind of row; the last rows
    and the whole in place."""
    x, res = randn(T, H, seed=1, dtype=BF16), randn(T, H, seed=2, scale=3.0, dtype=BF16)
    w = 1 + randn(H, seed=5, scale=0.3)
    xd, rd, wd = on(dev, x, res, w)
    say(f"[add_norm {T}x{H}]")
    out = moe.add_norm(xd, wd, residual=rd, eps=1e-5)
    for part in (slice(0, 40), slice(T - 40, T)):
        check_normed(moe.Normed(*(t[part] for t in out)), x[part], w, res[part], 1e-5, "rows")
    alone = moe.add_norm(xd[: T // 2], wd, residual=rd[: T // 2], eps=1e-5)     # half the rows: cached
    assert all(torch.equal(a, b[: T // 2]) for a, b in zip(alone, out))
    moe.add_norm(xd, wd, rd, 1e-5, out=moe.Normed(rd, xd, None, None))
    assert torch.equal(rd, out.h) and torch.equal(xd, out.y)


# ------------------------------------------------------------- gradients of the product

@pytest.mark.parametrize("M,N,K,act,dtype", [
    (1, 1, 128, "none", F32), (7, 384, 256, "none", F32), (65, 130, 128, "sigmoid", BF16), (129, 70, 384, "silu", BF16),
    (300, 384, 512, "relu", F32), (1000, 33, 256, "gelu", F32), (4100, 40, 256, "none", F32), (63, 1000, 128, "gelu", BF16),
    (200, 129, 640, "relu", BF16), (200, 129, 640, "none", BF16),
    # the tile shapes, the contraction split and not
    (128, 1000, 8192, "none", F32), (128, 12001, 1024, "none", F32), (2048, 16500, 768, "none", F32),
    (1000, 500, 8192, "silu", BF16), (12000, 500, 1024, "none", F32), (16500, 2000, 768, "none", F32),
    # the most columns, the longest rows
    (3, 65536, 128, "none", F32), (70, 65529, 256, "silu", BF16), (5, 20, 65536, "none", F32),
    # short contractions over 128, 256 and 384 columns of dz
    (5003, 100, 8064, "none", F32), (5001, 200, 8064, "silu", BF16), (4997, 300, 8064, "none", F32), (20001, 384, 1152, "none", F32)])
def test_linear_grad_keeps_dz(dev, M, N, K, act, dtype):
    """dx and dw are off by their own rounding and by 2^-15 of dz (a bf16 dz would add 2^-8
    of it), whatever dy's type and the activation."""
    x, w = randn(M, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=1 / math.sqrt(K), dtype=BF16)
    dy = randn(M, N, seed=3, dtype=dtype)
    z = None if act == "none" else randn(M, N, seed=4, scale=1.5)
    say(f"[linear_grad {M}x{N}x{K} {act} {dtype}]")
    dx, dw, _ = moe.linear_grad(*on(dev, dy, x, w), act=act, z=None if z is None else z.to(dev))
    torch.cuda.synchronize()
    rdx, rdw, _, dz = ob.linear_grad_ref(dy, x, w, act, z)
    op = 2.0 ** -15 + (0 if act == "none" else 32 * U)       # the operand's two parts, its slope
    ax, aw = dz.abs() @ w.to(F64).abs(), dz.abs().t() @ x.to(F64).abs()
    within(dx, rdx, rdx.abs() * BF + ax * (op + (2 * N / 32 + 64) * 2 * U), "dx")
    within(dw, rdw, rdw.abs() * BF + aw * (op + (2 * M / 32 + 64) * 2 * U), "dw")


def test_linear_grad_of_infinities_and_far_values(dev):
    """An infinite dy reaches its own row of dx and its own row of dw, as an infinity (its
    low part is 0); values near fp32's largest stay finite in both parts."""
    M, N, K = 70, 40, 128
    x, w = randn(M, K, seed=1, dtype=BF16).abs() + 1, randn(N, K, seed=2, dtype=BF16).abs() + 1
    dy = randn(M, N, seed=3)
    dy[3, 5], dy[9, 7] = math.inf, -math.inf
    dy[20] = 0
    dy[20, 11] = 3.3999e38                       # above bf16's largest value
    w[11] = 2.0 ** -10
    x[20] = 2.0 ** -10
    dx, dw, _ = (t.cpu() for t in moe.linear_grad(*on(dev, dy, x, w)))
    assert bool((dx[3] == math.inf).all()) and bool((dx[9] == -math.inf).all())
    assert bool((dw[5] == math.inf).all()) and bool((dw[7] == -math.inf).all())
    rows = [m for m in range(M) if m not in (3, 9)]
    cols = [n for n in range(N) if n not in (5, 7)]
    assert bool(torch.isfinite(dx[rows]).all()) and bool(torch.isfinite(dw[cols]).all())
    rdx = ob.linear_grad_ref(dy[rows], x[rows], w)[0]
    within(dx[rows], rdx, rdx.abs() * BF + (dy[rows].abs().to(F64) @ w.to(F64)) * 2.0 ** -14, "dx")


def test_linear_grad_in_two_parts_past_32_bits(dev, room):
    """dz's high and low parts at offsets past 2^32 bytes, read along its rows and transposed."""
    M, N, K, n = 1048579, 2056, 128, 70
    x, w, dy = randn(n, K, seed=1, dtype=BF16), randn(N, K, seed=2, scale=0.1, dtype=BF16), randn(n, N, seed=3)
    say(f"[linear_grad {M}x{N}x{K} float32]")
    dx, dw, db = moe.linear_grad(tail_rows(dev, M, N, dy, dtype=F32), tail_rows(dev, M, K, x, fill=1.0), w.to(dev))
    rdx, rdw, rdb, dz = ob.linear_grad_ref(dy, x, w)
    ax, aw = dz.abs() @ w.to(F64).abs(), dz.abs().t() @ x.to(F64).abs()
    within(dx[-n:], rdx, rdx.abs() * BF + ax * (2.0 ** -15 + (2 * N / 32 + 64) * 2 * U), "dx")
    assert not bool(dx[:1000].any())
    within(dw, rdw, rdw.abs() * BF + aw * (2.0 ** -15 + (2 * n / 32 + 64) * 2 * U), "dw")
    within(db, rdb, dz.abs().sum(0) * (n + 64) * U, "dbias")


@pytest.mark.parametrize("M", [1, 2, 4, 5, 8])
@pytest.mark.parametrize("N,K", [(384, 128), (17, 512), (385, 1024), (769, 7168), (512, 7168), (1024, 4096), (2048, 3584),
                                 (2047, 1024), (2049, 1024), (3, 65536), (1500, 8192)])
def test_linear_of_few_rows_on_both_sides_of_the_choice(dev, M, N, K):
    check_linear(dev, M, N, K, dtype=F32 if N % 2 else BF16, bias=K < 4096, res=N == 385, seed=M + N)


def test_sigmoid_slope_keeps_its_digits(dev):
    """One row of dy = 1: dbias is the slope itself, e^-|z| / (1 + e^-|z|)^2, to a few roundings
    at either end."""
    z = torch.linspace(-60, 60, 1201).view(1, -1)
    N = z.shape[1]
    x, w = torch.ones(1, 128, dtype=BF16), torch.ones(N, 128, dtype=BF16)
    e = torch.exp(-z.to(F64).abs())
    want = (e / (1 + e) ** 2)[0]
    for dtype in (BF16, F32):
        _, _, db = moe.linear_grad(*on(dev, torch.ones(1, N, dtype=dtype), x, w), act="sigmoid", z=z.to(dev))
        within(db, want, want * 16 * U, "slope")


# --------------------------------------------------------------------------- balance loss

@pytest.mark.parametrize("T,E", [(64, 384), (40, 512), (33, 300), (128, 512), (129, 512), (256, 256), (512, 100), (512, 256),
                                 (300, 385)])
@pytest.mark.parametrize("score", SCORES)
def test_balance_loss_of_small_batches(dev, T, E, score):
    """On both sides of the choice between one workgroup and four launches."""
    l = randn(T, E, seed=T + E, scale=1.5)
    ids = torch.randint(-1, E + 1, (T, 6), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    say(f"[balance {T}x{E} {score}]")
    check_balance(dev, l, ids, 0.3, score, None, "one sequence")
    check_balance(dev, l.to(BF16), ids, 0.3, score, [1, T // 3, T // 3, T - 5], "sequences, bf16")
    check_balance(dev, l, ids, 0.3, score, [0, T // 4, T // 3, T // 2, T - 1], "four sequences")


@pytest.mark.parametrize("T,E", [(40, 64), (600, 384), (30, 450), (9, 1000), (5, 4096)])
@pytest.mark.parametrize("score", ["sigmoid", "sqrtsoftplus"])
def test_balance_loss_of_rows_with_tiny_scores(dev, T, E, score):
    """Rows whose scores fp32 cannot hold have their probabilities and gradient all the same,
    down to logits of -690."""
    l = randn(T, E, seed=T, scale=1.5)
    for i, shift in enumerate((-30.0, -39.0, -42.0, -60.0, -88.0, -100.0, -175.0, -300.0, -680.0)):
        l[i::11] += shift
    l[2::11, 1::3] = -math.inf
    ids = torch.randint(0, E, (T, 6), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    say(f"[balance {T}x{E} {score}]")
    for logits in (l, l.to(BF16)):
        check_balance(dev, logits, ids, 0.3, score, None, "tiny scores")
        check_balance(dev, logits, ids, 0.3, score, [1, T // 3, T // 3, T - 1], "tiny scores, sequences")
    l[:] = -800.0                                  # below the documented end: no probabilities
    loss, _, dl = moe.balance_loss(*on(dev, l, ids), 0.3, score=score)
    assert float(loss) == 0 and not bool(dl.any())


def guarded(nbytes, dev):
    """(device address of nbytes between guards, check): check fails where a guard byte
    changed."""
    room = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device=dev)
    start = 4096 + (-(room.data_ptr() + 4096)) % 256

    def check(what):
        assert bool((room[:start] == 0xA5).all()) and bool((room[start + nbytes:] == 0xA5).all()), what
    return room.data_ptr() + start, check


@pytest.mark.parametrize("T,E,B", [(100, 16, 3), (100, 30, 5), (100, 16, 300), (1000, 24, 2), (1000, 384, 40), (700, 600, 400)])
@pytest.mark.parametrize("score", [0, 1, 2])
def test_balance_loss_of_unordered_offsets_writes_its_buffers_only(dev, T, E, B, score):
    """Every way to find a token's sequence, in one workgroup and in four launches, with
    offsets that run up and down and past both ends: the values are unspecified, what lies
    around the outputs and the workspace stays."""
    g = torch.Generator().manual_seed(B)
    l, ids = randn(T, E, seed=1).to(dev), torch.randint(-3, E + 3, (T, 4), generator=g, dtype=torch.int32).to(dev)
    far = torch.tensor([2 ** 31 - 1, -2 ** 31, T + 1, -1], dtype=torch.int64)
    d = moe.GateDims(T, E, 4, score, 0, 1, 1.0)
    nbytes = moe.lib().moe_balance_loss_workspace_bytes(d, B)
    for turn in range(4):
        off = torch.randint(-50, T + 50, (B + 1,), generator=g)
        if turn % 2:
            at = torch.randint(0, B + 1, (3,), generator=g)
            off[at] = far[torch.randint(0, 4, (3,), generator=g)]
        if turn == 3:
            off = off.flip(0).sort(descending=True).values
        off = off.clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).to(dev)
        say(f"[balance unordered {T}x{E} B={B} score {score} turn {turn}]")
        bufs = [guarded(n, dev) for n in (4, 4 * B * E, 4 * T * E, nbytes)]
        torch.cuda.synchronize()
        rc = moe.lib().moe_balance_loss(d, B, 1.0, l.data_ptr(), ids.data_ptr(), off.data_ptr(), bufs[0][0], bufs[1][0],
                                        bufs[2][0], bufs[3][0] if nbytes else None, nbytes, None)
        torch.cuda.synchronize()
        assert rc == moe.MOE_OK
        for (_, check), name in zip(bufs, ("loss", "counts", "d_logits", "ws")):
            check(name)


# ----------------------------------------------------------------------------------- gate

FAR_BIASES = [1e3, -1e3, -1e4, -1e9, 1e9, -3e38, 3e38, -math.inf, math.inf, math.nan]


@pytest.mark.parametrize("T,E,K", [(20, 384, 8), (33, 37, 5), (9, 600, 17), (4, 2100, 64)])
@pytest.mark.parametrize("score", SCORES)
def test_gate_with_far_biases(dev, T, E, K, score):
    """Experts forced in or held back by biases of any size leave the others' choice exact,
    near ties of the others among them."""
    l = randn(T, E, seed=E, scale=2.0)
    l[:, 1::4] = l[:, 0::4][:, : l[:, 1::4].shape[1]] + 1e-7       # pairs that fp32 scores cannot tell apart
    l[3, E // 2:] = -math.inf
    say(f"[gate {T}x{E} top-{K} {score}]")
    for far in FAR_BIASES:
        b = randn(E, seed=3, scale=0.1)
        b[0::4] = 0.0
        b[1::4] = 0.0
        b[7] = far
        check_gate(dev, l, K, f"one bias of {far}", score, bias=b)
        b[2::3] = far
        check_gate(dev, l, K, f"a third of the biases {far}", score, bias=b)
        b[: E - 3] = far                                           # fewer than K left where they are held back
        check_gate(dev, l, K, f"most biases {far}", score, bias=b)


@pytest.mark.parametrize("score", SCORES)
def test_gate_is_not_slowed_by_far_biases(dev, score):
    """One expert held back or forced in by a finite bias leaves the fast path to the rows
    (ranking every row in 64 bits takes ten to twenty times as long)."""
    l = randn(8192, 384, seed=1).to(dev)

    def us(far):
        b = randn(384, seed=2, scale=0.1)
        if far:
            b[17] = far
        bd = b.to(dev)
        best = math.inf
        for _ in range(5):
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(40):
                moe.gate(l, 8, score=score, bias=bd)
            torch.cuda.synchronize()
            best = min(best, (time.perf_counter() - t) / 40 * 1e6)
        return best
    plain = us(None)
    for far in (-1e4, -1e9, 1e9, torch.finfo(F32).min):
        t = us(far)
        say(f"[gate {score}] bias {far}: {t:.1f} us against {plain:.1f}")
        assert t < 3 * plain


def test_unaligned_scalars_are_refused_by_name(dev):
    """One counter out of several starts at any multiple of 4 bytes: the error says so."""
    l, counters = randn(4, 8, seed=1).to(dev), torch.tensor([0, 4, 0, 0, 4], dtype=torch.int32, device=dev)
    with pytest.raises(moe.MoEError, match="16-byte aligned") as e:
        moe.gate(l, 2, n_valid=counters[1:2])
    assert hex(counters[1:2].data_ptr()) in str(e.value)
    ids, _ = moe.gate(l, 2, n_valid=counters[4:5])
    with pytest.raises(moe.MoEError, match="16-byte aligned"):
        moe.balance_loss(l, ids, 1.0, seq_offsets=counters[:2].clone().repeat(2)[2:])
    with pytest.raises(moe.MoEError, match="16-byte aligned"):
        moe.gate(l, 2, topk_weights=torch.empty(9, device=dev)[1:].view(4, 2))
    with pytest.raises(moe.MoEError) as e:
        moe.balance_loss(l, ids, math.nan)
    assert "aligned" not in str(e.value)
