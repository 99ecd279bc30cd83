"""Cases of the operators that train the routed experts, for measuring: tokens laid out by expert (``sort``) and brought
back with their weights (``return``), the experts' products on rows grouped by expert (``experts``), and the gated
activation between them with its input saved in 8 bits (``glu``), with their gradients.

``run`` computes a case in plain torch (``own`` false) or by the framework's calls (``own`` true); ``exact`` computes
the same outputs in 64 bits. Sizes are those of the framework's own workloads (hidden 7168, 384 experts, top-8, one
rank's intermediate slice of 384, 7 to 32768 tokens) and of the ranges around them.
"""

import math

import torch

own = False

ACTS = ("silu", "gelu", "relu", "sigmoid", "none")


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the 7-token verify step: 56 rows, bound by latency
        dict(name="sort_verify7", op="sort", T=7, H=7168, E=384, K=8, skew=1.0, drop=False, codes=False),
        # a 32K chunk: one read of the activation, eight writes of it
        dict(name="sort_prefill32k", op="sort", T=32768, H=7168, E=384, K=8, skew=1.2, drop=False, codes=False),
        # the backward pass of a training step lays its rows out again, from the 8-bit codes that were kept
        dict(name="sort_saved16k", op="sort", T=16383, H=7168, E=384, K=8, skew=0.4, drop=True, codes=True),
        # a decode step of 256 tokens brings its rows back onto a shared expert's output
        dict(name="return_decode256", op="return", T=256, H=7168, E=384, K=8, skew=1.1, drop=False, weighted=True,
             add=True, f32=False),
        # a 32K chunk brought back
        dict(name="return_prefill32k", op="return", T=32768, H=7168, E=384, K=8, skew=1.2, drop=False, weighted=True,
             add=False, f32=False),
        # the gradient of that in a training step of an odd number of tokens, some picks dropped
        dict(name="return_grad8k", op="return_grad", T=8191, H=7168, E=384, K=8, skew=0.4, drop=True, f32=False),
        # gate and up products of the 7-token verify: the weights of about 50 experts stream by, a row or two each
        dict(name="experts_verify7", op="experts", T=7, E=384, K=8, skew=1.0, drop=False, N=768, C=7168, f32=False),
        # gate and up products of a 32K chunk, experts of a few rows beside one that nearly every token picks
        dict(name="experts_prefill32k", op="experts", T=32768, E=384, K=8, skew=1.2, drop=False, N=768, C=7168,
             f32=False),
        # input and weight gradients of a training step under a balance loss
        dict(name="experts_grad8k", op="experts_grad", T=8191, E=384, K=8, skew=0.4, drop=True, N=768, C=7168,
             f32=False),
        # the smallest model's batch of 64 tokens
        dict(name="glu_64", op="glu", T=64, E=8, K=2, skew=0.0, drop=False, I=512, act="silu"),
        # the activation of a 32K chunk, its input saved for the backward pass
        dict(name="glu_prefill32k", op="glu", T=32768, E=384, K=8, skew=1.2, drop=False, I=384, act="silu"),
        # the backward pass from the saved codes, rows of dropped picks behind the last expert's
        dict(name="glu_grad32k", op="glu_grad", T=32768, E=384, K=8, skew=0.4, drop=True, I=384, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sort", "sort", "return", "return", "return_grad", "experts", "experts", "experts_grad", "glu",
                     "glu_grad"))
    E = _log(rng, 1, 512)
    K = rng.randint(1, min(E, 12))
    c = dict(op=op, E=E, K=K, skew=round(rng.uniform(0.0, 1.3), 2), drop=rng.random() < 0.4)
    if op in ("sort", "return", "return_grad"):
        c["H"] = 8 * _log(rng, 1, 2048)
        if op == "sort":
            c["codes"] = rng.random() < 0.4
            if c["codes"]:
                c["H"] = 128 * _log(rng, 1, 128)
        else:
            c["f32"] = rng.random() < 0.3
        if op == "return":
            c["weighted"], c["add"] = rng.random() < 0.7, rng.random() < 0.4
        most = 32768 * 8 * 7168 // (c["H"] * K) // (4 if op == "return_grad" else 2)
    elif op in ("glu", "glu_grad"):
        c["I"] = 128 * _log(rng, 1, 32)
        c["act"] = rng.choice(ACTS)
        most = 32768 * 8 * 384 // (c["I"] * K)
    else:
        c["N"], c["C"] = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 56)
        c["f32"] = rng.random() < 0.3
        # fewer experts where each has many weights
        c["E"] = max(1, min(E, (1 << 30) // (c["N"] * c["C"])))
        c["K"] = min(K, c["E"])
        most = 2 ** 38 // (c["N"] * c["C"] * c["K"]) // (2 if op == "experts_grad" else 1)
    c["T"] = _log(rng, 1, max(1, min(65536, most)))
    return c


# ------------------------------------------------------------------------------------------------------------ inputs

def _route(case, g, dev):
    """Picks of a router whose experts' popularity falls off as rank^-skew, and the plan that sorts them by expert:
    offsets of the experts' rows, pairs in the order of their rows, the row of every pair (-1: dropped)."""
    T, E, K = case["T"], case["E"], case["K"]
    rank = torch.randperm(E, generator=g, device=dev).float() + 1
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
    ids = torch.topk(noise - case["skew"] * torch.log(rank), K, dim=1).indices
    if case["drop"]:
        gone = torch.rand(T, K, generator=g, device=dev) < 0.02
        gone[0, 0] = False                                  # one row at least
        ids[gone] = -1
    e = torch.where(ids < 0, E, ids).reshape(-1)
    pairs = torch.sort(e, stable=True).indices
    counts = torch.bincount(e, minlength=E + 1)[:E]
    off = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    off[1:] = counts.cumsum(0)
    live = int(off[-1])
    rows = torch.full((T * K,), -1, dtype=torch.int64, device=dev)
    rows[pairs[:live]] = torch.arange(live, device=dev)
    pairs[live:] = -1
    return {"ids": ids.int(), "off": off.int(), "pairs": pairs.int(), "rows": rows.int(), "live": live,
            "sizes": counts.tolist()}


def _codes(x):
    """E4M3 codes and E8M0 scales of the columns of x in blocks of 128, the smallest scale that fits each block."""
    R, C = x.shape
    blocks = x.float().view(R, C // 128, 128)
    m, e = torch.frexp(blocks.abs().amax(2))                # amax = m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-127)   # smallest e with amax <= 448 * 2^e
    q = torch.ldexp(blocks, -e[:, :, None]).view(R, C).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 29)
    bf = torch.bfloat16

    def normal(*shape, scale=1.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    def buffer(*shape, dtype=bf):
        """A program's own buffer: rows behind the last expert's stay as they are."""
        return torch.zeros(*shape, dtype=dtype, device=dev)

    s = dict(case)
    s.update(_route(case, g, dev))
    op, T, E, P, live = case["op"], case["T"], case["E"], case["T"] * case["K"], s["live"]
    f = torch.float32 if case.get("f32") else bf
    if op == "sort":
        x = normal(T, case["H"])
        if case["codes"]:
            s["x_q"], s["x_s"] = _codes(x)
        else:
            s["x"] = x
        s["out"] = buffer(P, case["H"])
    elif op == "return":
        s["x"] = normal(P, case["H"])
        s["w"] = torch.rand(T, case["K"], generator=g, device=dev) if case["weighted"] else None
        s["add"] = normal(T, case["H"], dtype=f) if case["add"] else None
    elif op == "return_grad":
        s["x"], s["dy"] = normal(P, case["H"]), normal(T, case["H"], dtype=f)
        s["w"] = torch.rand(T, case["K"], generator=g, device=dev)
        s["out"] = buffer(P, case["H"])
    elif op in ("experts", "experts_grad"):
        N, C = case["N"], case["C"]
        s["x"] = normal(P, C)
        s["weight"] = torch.empty(E, N, C, dtype=bf, device=dev)
        s["weight"].normal_(0.0, 1 / math.sqrt(C), generator=g)
        if op == "experts":
            s["out"] = buffer(P, N, dtype=f)
        else:
            s["dy"], s["out"] = normal(P, N), buffer(P, C)
    else:
        z = normal(P, 2 * case["I"], scale=1.5)
        if op == "glu":
            s["z"] = z
            s["h"] = buffer(P, case["I"])
            s["z_q"] = buffer(P, 2 * case["I"], dtype=torch.uint8)
            s["z_s"] = buffer(P, 2 * case["I"] // 128, dtype=torch.uint8)
        else:
            s["z_q"], s["z_s"] = _codes(z)
            s["dh"], s["h"], s["dz"] = normal(P, case["I"]), buffer(P, case["I"]), buffer(P, 2 * case["I"])
    return s


# ------------------------------------------------------------------------------------------- the operators, own calls

def _plan(moe, s):
    """The plan as the framework's handle, kept with its tensors as a program keeps it over a step's calls."""
    if "plan" not in s:
        empty = torch.empty(1, dtype=torch.int32, device=s["off"].device)
        s["plan"] = moe.Plan(moe.make_dims(s["T"], 128, 128, s["E"], s["K"]), s["off"], s["pairs"], s["rows"], empty,
                             empty)
    return s["plan"]


def _own(s):
    import mxfp4_weights_fp8_amd as moe
    op, p = s["op"], _plan(moe, s)
    u8 = torch.uint8
    if op == "sort":
        if s["codes"]:
            return moe.sort_rows(s["x_q"].view(u8), p, scales=s["x_s"].view(u8), rows=s["out"])
        return moe.sort_rows(s["x"], p, rows=s["out"])
    if op == "return":
        return moe.return_rows(s["x"], p, weights=s["w"], add=s["add"],
                               dtype=torch.float32 if s["f32"] else torch.bfloat16)
    if op == "return_grad":
        d_rows, d_weights = moe.return_rows_grad(s["dy"], s["x"], p, s["w"], d_rows=s["out"])
        return {"d_rows": d_rows, "d_weights": d_weights}
    f = torch.float32 if s.get("f32") else torch.bfloat16
    if op == "experts":
        return moe.expert_linear(s["x"], s["weight"], p, dtype=f, y=s["out"])
    if op == "experts_grad":
        dx, dw = moe.expert_linear_grad(s["dy"], s["x"], s["weight"], p, dtype=f, dx=s["out"])
        return {"dx": dx, "dw": dw}
    if op == "glu":
        h, z_q, z_s = moe.glu(s["z"], act=s["act"], p=p, out=(s["h"], s["z_q"], s["z_s"]))
        return {"h": h, "z_q": z_q.view(torch.float8_e4m3fn), "z_s": z_s.view(torch.float8_e8m0fnu)}
    dz, h = moe.glu_grad(s["dh"], s["z_q"].view(u8), scales=s["z_s"].view(u8), act=s["act"], p=p,
                         out=(s["dz"], s["h"]))
    return {"dz": dz, "h": h}


# ------------------------------------------------------------------------------------------- the operators, plain form

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return torch.sigmoid(z) if act == "sigmoid" else z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "sigmoid":
        p = torch.sigmoid(z)
        return p * (1 - p)
    return torch.ones_like(z)


def _values(q, s):
    """What codes and their scales stand for."""
    R, C = q.shape
    e = s.view(torch.uint8).int() - 127
    return torch.ldexp(q.float().view(R, C // 128, 128), e[:, :, None]).view(R, C)


def _blocks(s):
    """The live rows in blocks of one expert's rows: the place of every row in them, and the expert of every block. The
    number of blocks is known on the host from the plan."""
    size = min(256, max(1, s["live"] // s["E"]))
    off = s["off"].long()
    per = (off[1:] - off[:-1] + size - 1) // size           # blocks of each expert
    count = sum((n + size - 1) // size for n in s["sizes"])
    first = per.cumsum(0) - per
    r = torch.arange(s["live"], device=off.device)
    e = torch.searchsorted(off, r, right=True) - 1
    at = first[e] * size + r - off[e]
    expert = torch.repeat_interleave(torch.arange(s["E"], device=off.device), per, output_size=count)
    return size, count, at, expert


def _in_blocks(x, at, size, count):
    return torch.zeros(count * size, x.shape[1], device=x.device).index_copy_(0, at, x[:at.numel()].float()).view(
        count, size, x.shape[1])


def _behind(live, like, v):
    """v's live rows on top of what a program's buffer holds behind them."""
    out = torch.zeros_like(like)
    out[:live] = v[:live].to(like.dtype)
    return out


def _plain(s):
    op, live, bf = s["op"], s["live"], torch.bfloat16
    if op == "sort":
        x = _values(s["x_q"], s["x_s"]).to(bf) if s["codes"] else s["x"]
        return _behind(live, s["out"], x[s["pairs"][:live].long() // s["K"]])
    if op in ("return", "return_grad"):
        T, K = s["T"], s["K"]
        at = s["rows"].long()
        rows = s["x"][at.clamp(min=0)].float() * (at >= 0)[:, None]       # the rows of every token's picks, 0 for none
        rows = rows.view(T, K, -1)
        if op == "return_grad":
            dy = s["dy"].float()
            t = s["pairs"][:live].long()
            d_rows = s["w"].reshape(-1)[t, None] * dy[t // K]
            return {"d_rows": _behind(live, s["out"], d_rows), "d_weights": (rows * dy[:, None]).sum(2)}
        if s["w"] is not None:
            rows = rows * s["w"][:, :, None]
        y = rows.sum(1)
        if s["add"] is not None:
            y = y + s["add"].float()
        return y if s["f32"] else y.to(bf)
    if op in ("experts", "experts_grad"):
        f = torch.float32 if s["f32"] else bf
        size, count, at, expert = _blocks(s)
        x = _in_blocks(s["x"], at, size, count)
        if op == "experts":
            y = torch.bmm(s["weight"][expert].float(), x.transpose(1, 2).contiguous()).transpose(1, 2)
            return _behind(live, s["out"], y.reshape(count * size, -1)[at])
        dy = _in_blocks(s["dy"], at, size, count)
        dx = torch.bmm(dy, s["weight"][expert].float()).view(count * size, -1)[at]
        dw = torch.zeros(s["weight"].shape, device=x.device).index_add_(0, expert, torch.bmm(
            dy.transpose(1, 2).contiguous(), x))
        return {"dx": _behind(live, s["out"], dx), "dw": dw.to(f)}
    I = s["I"]
    if op == "glu":
        z = s["z"].float()
        q, scale = _codes(z)
        h = _act(z[:, :I], s["act"]) * z[:, I:]
        u8 = torch.uint8
        return {"h": _behind(live, s["h"], h), "z_q": _behind(live, s["z_q"], q.view(u8)).view(torch.float8_e4m3fn),
                "z_s": _behind(live, s["z_s"], scale.view(u8)).view(torch.float8_e8m0fnu)}
    z, dh = _values(s["z_q"], s["z_s"]), s["dh"].float()
    gate, up = z[:, :I], z[:, I:]
    a = _act(gate, s["act"])
    dz = torch.cat([dh * up * _act_slope(gate, s["act"]), dh * a], 1)
    return {"dz": _behind(live, s["dz"], dz), "h": _behind(live, s["h"], a * up)}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------------------------- work

def _expected(case):
    """Rows of picks that are not dropped, and experts that have any, as expected of the distribution."""
    T, E, K = case["T"], case["E"], case["K"]
    weight = [(i + 1.0) ** -case["skew"] for i in range(E)]
    total = sum(weight)
    picked = sum(1 - (1 - min(1.0, w / total)) ** (T * K) for w in weight)
    return int(T * K * (0.98 if case["drop"] else 1.0)), max(1, min(T * K, int(picked)))


def work(case):
    op, T, P = case["op"], case["T"], case["T"] * case["K"]
    rows, experts = _expected(case)
    f = 4 if case.get("f32") else 2
    if op == "sort":
        H = case["H"]
        return {"bytes": T * H * (1 + 1 / 128 if case["codes"] else 2) + rows * H * 2 + 4 * P, "flops": 0}
    if op == "return":
        H = case["H"]
        return {"bytes": rows * H * 2 + T * H * f * (2 if case["add"] else 1) + P * (8 if case["weighted"] else 4),
                "flops": 2 * rows * H}
    if op == "return_grad":
        H = case["H"]
        return {"bytes": rows * H * 4 + T * H * f + 12 * P, "flops": 3 * rows * H}
    if op == "experts":
        N, C = case["N"], case["C"]
        return {"bytes": rows * (2 * C + f * N) + 2 * experts * N * C, "flops": 2 * rows * N * C}
    if op == "experts_grad":
        N, C = case["N"], case["C"]
        return {"bytes": rows * (2 * C + 2 * N + 2 * C) + 2 * experts * N * C + f * case["E"] * N * C,
                "flops": 4 * rows * N * C}
    I = case["I"]
    z8 = rows * 2 * I * (1 + 1 / 128)
    if op == "glu":
        return {"bytes": rows * 6 * I + z8, "flops": 16 * rows * I}
    return {"bytes": rows * 8 * I + z8, "flops": 24 * rows * I}


# ------------------------------------------------------------------------------------------------- the exact outputs

def exact(case, seed):
    s = prepare(case, seed)
    op, T, E, K, live = case["op"], case["T"], case["E"], case["K"], s["live"]
    d = torch.float64
    off = s["off"].tolist()
    ids = s["ids"].long().reshape(-1)

    def decoded(q, scale):
        return q.to(d) * torch.exp2(scale.view(torch.uint8).to(d) - 127).repeat_interleave(128, 1)

    def sorted_pairs():
        """Pairs expert by expert, in rising order within one."""
        return torch.argsort(torch.where(ids < 0, E, ids) * ids.numel() + torch.arange(ids.numel(), device=ids.device))

    def whole(v, width, dtype=d):
        """Rows behind the last expert's are the buffer's zeros."""
        out = torch.zeros(T * K, width, dtype=dtype, device=v.device)
        out[:live] = v[:live]
        return out

    if op == "sort":
        token = sorted_pairs()[:live] // K
        if case["codes"]:
            return whole(decoded(s["x_q"], s["x_s"])[token], case["H"])
        return whole(s["x"][token].to(d), case["H"])
    if op in ("return", "return_grad"):
        pairs = sorted_pairs()[:live]
        token = pairs // K
        if op == "return":
            y = torch.zeros(T, case["H"], dtype=d, device=pairs.device) if s["add"] is None else s["add"].to(d)
            w = torch.ones(T * K, dtype=d, device=pairs.device) if s["w"] is None else s["w"].to(d).reshape(-1)
            for lo in range(0, live, 1 << 16):
                hi = min(live, lo + (1 << 16))
                y.index_add_(0, token[lo:hi], s["x"][lo:hi].to(d) * w[pairs[lo:hi], None])
            return y
        d_rows = whole(s["dy"].to(d)[token] * s["w"].to(d).reshape(-1)[pairs, None], case["H"])
        d_weights = torch.zeros(T * K, dtype=d, device=pairs.device)
        for lo in range(0, live, 1 << 16):
            hi = min(live, lo + (1 << 16))
            d_weights[pairs[lo:hi]] = torch.einsum("rh,rh->r", s["x"][lo:hi].to(d), s["dy"][token[lo:hi]].to(d))
        return {"d_rows": d_rows, "d_weights": d_weights.view(T, K)}
    if op in ("experts", "experts_grad"):
        N, C = case["N"], case["C"]
        out = torch.zeros(T * K, N if op == "experts" else C, dtype=d, device=ids.device)
        dw = torch.zeros(E, N, C, dtype=d, device=ids.device) if op == "experts_grad" else None
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                w, x = s["weight"][e].to(d), s["x"][lo:hi].to(d)
                if op == "experts":
                    out[lo:hi] = torch.mm(x, w.t())
                else:
                    dy = s["dy"][lo:hi].to(d)
                    out[lo:hi] = torch.mm(dy, w)
                    dw[e] = torch.mm(dy.t(), x)
        return out if op == "experts" else {"dx": out, "dw": dw}
    act, I = case["act"], case["I"]

    def sigma(v):
        return 1 / (1 + torch.exp(-v))

    def cdf(v):
        return torch.special.ndtr(v)

    def value(v):
        return {"none": lambda: v, "relu": lambda: torch.where(v > 0, v, 0.0), "silu": lambda: v * sigma(v),
                "gelu": lambda: v * cdf(v), "sigmoid": lambda: sigma(v)}[act]()

    def slope(v):
        return {"none": lambda: torch.ones_like(v), "relu": lambda: torch.where(v > 0, 1.0, 0.0).to(d),
                "silu": lambda: sigma(v) + v * sigma(v) * sigma(-v),
                "gelu": lambda: cdf(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi),
                "sigmoid": lambda: sigma(v) * sigma(-v)}[act]()

    if op == "glu":
        z = s["z"].to(d)
        top = z.abs().view(T * K, -1, 128).max(2).values
        e = torch.ceil(torch.log2(top / 448).clamp(min=-127))
        # a code's value before its rounding to 8 bits; a scale is a power of two, all or nothing
        return {"h": whole(value(z[:, :I]) * z[:, I:], I),
                "z_q": whole(z / torch.exp2(e).repeat_interleave(128, 1), 2 * I), "z_s": None}
    z, dh = decoded(s["z_q"], s["z_s"]), s["dh"].to(d)
    dz = torch.cat([dh * z[:, I:] * slope(z[:, :I]), dh * value(z[:, :I])], 1)
    return {"dz": whole(dz, 2 * I), "h": whole(value(z[:, :I]) * z[:, I:], I)}
