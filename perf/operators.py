"""Cases of the operators around the routed FFN, for measuring: the residual add with RMS norm and 8-bit output
(``add_norm``), the dense product with its epilogue (``linear``), the router's gate (``gate``) and the balance loss
(``balance_loss``), each with its gradient.

``run`` computes a case in plain torch (``own`` false) or by the framework's calls (``own`` true); ``exact`` computes
the same outputs in 64 bits. Sizes are those of the framework's own workloads (hidden 7168, 384 experts, top-8, 7 to
32768 tokens) and of the ranges around them.
"""

import math

import torch

own = False

EPS = 1e-6
SUM_EPS = 1e-20       # added to the sum of the chosen scores before the division
ACTS = ("none", "relu", "silu", "gelu", "sigmoid")
SCORES = ("softmax", "sigmoid", "sqrtsoftplus")


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the 7-token verify step: one norm launch in front of the router and the experts, bound by latency
        dict(name="norm_verify7", op="norm", T=7, H=7168, residual=True, w32=False),
        # a 32K prefill chunk's residual add + norm + quantisation, bound by memory
        dict(name="norm_prefill32k", op="norm", T=32768, H=7168, residual=True, w32=False),
        # its backward pass in a router or norm tuning step of 4096 tokens and an odd remainder
        dict(name="norm_grad4k", op="norm_grad", T=4099, H=7168, dh=True, w32=True),
        # router product of the 7-token verify: 5.5 MB of weights, a few rows
        dict(name="router_verify7", op="linear", M=7, N=384, K=7168, act="none", bias=True, residual=False, f32=True),
        # router product of a 32K prefill chunk: reads the whole activation
        dict(name="router_prefill32k", op="linear", M=32768, N=384, K=7168, act="none", bias=False, residual=False,
             f32=True),
        # projection back to the hidden size with the residual's addition, an odd number of tokens
        dict(name="down_residual8k", op="linear", M=8191, N=7168, K=2048, act="none", bias=True, residual=True,
             f32=False),
        # the router's weight and input gradients from float32 logit gradients
        dict(name="router_grad16k", op="linear_grad", M=16384, N=384, K=7168, act="none", f32=True),
        # the gate of the 7-token verify: bias-corrected sigmoid scores
        dict(name="gate_verify7", op="gate", T=7, E=384, K=8, score="sigmoid", bias=True, renorm=True, pad=0,
             masked=False),
        # the gate of a prefill chunk with padding rows behind the last token
        dict(name="gate_prefill32k", op="gate", T=32768, E=384, K=8, score="sqrtsoftplus", bias=True, renorm=True,
             pad=100, masked=False),
        # its gradient, added to the gradient that the balance loss left
        dict(name="gate_grad32k", op="gate_grad", T=32768, E=384, K=8, score="softmax", renorm=True, add=True),
        # balance loss of a small batch of one sequence
        dict(name="balance_256", op="balance", T=256, E=64, K=6, B=1, score="softmax"),
        # balance loss over ragged sequences of a training batch, one of them empty, rows behind the last one
        dict(name="balance_ragged32k", op="balance", T=32768, E=384, K=8, B=17, score="sigmoid"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_grad", "linear", "linear", "linear_grad", "gate", "gate", "gate_grad",
                     "balance", "balance"))
    if op in ("norm", "norm_grad"):
        H = 128 * _log(rng, 1, 128)
        T = _log(rng, 1, max(1, min(65536, 32768 * 7168 // H)))
        if op == "norm":
            return dict(op=op, T=T, H=H, residual=rng.random() < 0.8, w32=rng.random() < 0.5)
        return dict(op=op, T=T, H=H, dh=rng.random() < 0.7, w32=rng.random() < 0.5)
    if op in ("linear", "linear_grad"):
        K, N = 128 * _log(rng, 1, 64), _log(rng, 1, 8192)
        M = _log(rng, 1, max(1, min(32768, (1 << 36) // (N * K))))
        if op == "linear":
            return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                        residual=rng.random() < 0.4, f32=rng.random() < 0.5)
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), f32=rng.random() < 0.5)
    E = _log(rng, 2, 1024)
    T, K = _log(rng, 1, max(1, min(65536, 32768 * 384 // E))), rng.randint(1, min(E, 16))
    score = rng.choice(SCORES)
    if op == "gate":
        return dict(op=op, T=T, E=E, K=K, score=score, bias=rng.random() < 0.6, renorm=rng.random() < 0.7,
                    pad=rng.randint(0, T // 4), masked=rng.random() < 0.3)
    if op == "gate_grad":       # one renormalised weight is 1 whatever its logit: two picks at least
        return dict(op=op, T=T, E=E, K=max(2, K), score=score, renorm=rng.random() < 0.7, add=rng.random() < 0.5)
    # with every expert picked by every token the balance gradient is zero: fewer picks than experts
    return dict(op=op, T=T, E=E, K=min(K, E - 1), B=_log(rng, 1, 64), score=score)


# ------------------------------------------------------------------------------------------------------------ inputs

def _logits(case, g, dev):
    """Router logits: a popularity offset per expert plus a per-token part."""
    T, E = case["T"], case["E"]
    return torch.randn(T, E, generator=g, device=dev) * 1.3 + 0.7 * torch.randn(E, generator=g, device=dev)


def _picks(logits, K):
    """Picks of a top-K of the logits, as a gate of an earlier step gave them, some dropped."""
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)
    bf = torch.bfloat16

    def normal(*shape, scale=1.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        s["x"] = normal(T, H)
        s["res"] = normal(T, H, scale=3.0) if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn(H, generator=g, device=dev)).to(torch.float32 if case["w32"] else bf)
    elif op == "norm_grad":
        T, H = case["T"], case["H"]
        s["dy"], s["h"] = normal(T, H), normal(T, H, scale=3.0)
        s["dh"] = normal(T, H) if case["dh"] else None
        s["w"] = (1 + 0.2 * torch.randn(H, generator=g, device=dev)).to(torch.float32 if case["w32"] else bf)
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["w"] = normal(M, K), normal(N, K, scale=1.5 / math.sqrt(K))
        s["b"] = normal(N, dtype=torch.float32) if case["bias"] else None
        s["res"] = normal(M, N, scale=2.0, dtype=torch.float32 if case["f32"] else bf) if case["residual"] else None
    elif op == "linear_grad":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["w"] = normal(M, K), normal(N, K, scale=1.5 / math.sqrt(K))
        s["dy"] = normal(M, N, dtype=torch.float32 if case["f32"] else bf)
        s["z"] = None if case["act"] == "none" else normal(M, N, scale=1.5, dtype=torch.float32)
    elif op == "gate":
        T, E = case["T"], case["E"]
        s["logits"] = _logits(case, g, dev)
        if case["masked"]:      # experts taken out of service for some tokens, one token without any
            s["logits"][torch.rand(T, E, generator=g, device=dev) < 0.3] = -math.inf
            s["logits"][T // 2] = -math.inf
        s["bias"] = 0.1 * torch.randn(E, generator=g, device=dev) if case["bias"] else None
        s["n"] = torch.tensor([T - case["pad"]], dtype=torch.int32, device=dev) if case["pad"] else None
    elif op == "gate_grad":
        s["logits"] = _logits(case, g, dev)
        s["ids"] = _picks(s["logits"], case["K"])
        s["dw"] = torch.randn(case["T"], case["K"], generator=g, device=dev)
        s["add"] = 0.01 * torch.randn(case["T"], case["E"], generator=g, device=dev) if case["add"] else None
    else:
        T, B = case["T"], case["B"]
        s["logits"] = _logits(case, g, dev)
        s["ids"] = _picks(s["logits"], case["K"])
        s["ids"][torch.rand(s["ids"].shape, generator=g, device=dev) < 0.01] = -1     # dropped picks
        if B > 1:
            cuts = (torch.rand(B + 1, generator=g, device=dev) * T).long().sort().values
            cuts[0] = 0
            cuts[B // 2 + 1] = cuts[B // 2]           # an empty sequence
            s["off"] = cuts.sort().values.to(torch.int32)
        else:
            s["off"] = None
    return s


# ------------------------------------------------------------------------------------------- the operators, own calls

def _own(s):
    import mxfp4_weights_fp8_amd as moe
    op = s["op"]
    if op == "norm":
        h, y, x_q, x_s = moe.add_norm(s["x"], s["w"], residual=s["res"], eps=EPS)
        return {"h": h, "y": y, "x_q": x_q.view(torch.float8_e4m3fn), "x_s": x_s.view(torch.float8_e8m0fnu)}
    if op == "norm_grad":
        dx, dw = moe.add_norm_grad(s["dy"], s["h"], s["w"], eps=EPS, dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "linear":
        return moe.linear(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["res"],
                          dtype=torch.float32 if s["f32"] else torch.bfloat16)
    if op == "linear_grad":
        dx, dw, db = moe.linear_grad(s["dy"], s["x"], s["w"], act=s["act"], z=s["z"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "gate":
        ids, w = moe.gate(s["logits"], s["K"], score=s["score"], bias=s["bias"], renorm=s["renorm"], scale=2.5,
                          n_valid=s["n"])
        return {"ids": ids, "w": w}
    if op == "gate_grad":
        return moe.gate_grad(s["logits"], s["ids"], s["dw"], score=s["score"], renorm=s["renorm"], scale=2.5,
                             add=s["add"])
    loss, counts, dlogits = moe.balance_loss(s["logits"], s["ids"], 0.5, score=s["score"], seq_offsets=s["off"])
    return {"loss": loss, "counts": counts, "dlogits": dlogits}


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
    p = torch.sigmoid(z)
    return p * (1 - p)


def _score(l, score):
    """Scores of logits; an expert at minus infinity scores nothing, also where a row has no other."""
    if score == "softmax":
        m = l.amax(1, keepdim=True).clamp(min=torch.finfo(l.dtype).min)
        e = torch.exp(l - m)
        return e / e.sum(1, keepdim=True).clamp(min=1e-30)
    if score == "sigmoid":
        return torch.sigmoid(l)
    return torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))


def _score_slope(l, s, score):
    """d score / d logit where a score depends on its own logit alone."""
    if score == "sigmoid":
        return s * (1 - s)
    return torch.sigmoid(l) / (2 * s)


def _plain(s):
    op = s["op"]
    bf = torch.bfloat16
    if op == "norm":
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
        T, H = y.shape
        blocks = y.view(T, H // 128, 128)
        m, e = torch.frexp(blocks.abs().amax(2))            # amax = m 2^e, m in [0.5, 1)
        e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-127)   # smallest e with amax <= 448 * 2^e
        q = torch.ldexp(blocks, -e[:, :, None]).view(T, H).to(torch.float8_e4m3fn)
        x_s = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        return {"h": h.to(bf) if s["res"] is not None else s["x"], "y": y.to(bf), "x_q": q, "x_s": x_s}
    if op == "norm_grad":
        h, dy = s["h"].float(), s["dy"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n, g = h * r, dy * s["w"].float()
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(bf), "dw": (dy * n).sum(0)}
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return y if s["f32"] else y.to(bf)
    if op == "linear_grad":
        dz = s["dy"].float()
        if s["act"] != "none":
            dz = dz * _act_slope(s["z"], s["act"])
        return {"dx": (dz @ s["w"].float()).to(bf), "dw": (dz.t() @ s["x"].float()).to(bf), "db": dz.sum(0)}
    l, K = s["logits"], s["K"]
    if op == "gate":
        if s["bias"] is None:
            key = l                                         # scores rise with their logits
        else:                                               # 64 bits: keys that lie next to each other
            key = _score(l.double(), s["score"]) + s["bias"].double()
            key = torch.where(l > -math.inf, key, -math.inf)
        top, ids = torch.sort(key, dim=1, descending=True, stable=True)
        top, ids = top[:, :K], ids[:, :K]
        live = top > -math.inf
        if s["n"] is not None:
            live = live & (torch.arange(l.shape[0], device=l.device) < s["n"])[:, None]
        w = torch.where(live, _score(l, s["score"]).gather(1, ids), 0.0)
        if s["renorm"]:
            w = w / (w.sum(1, keepdim=True) + SUM_EPS)
        return {"ids": torch.where(live, ids, -1).to(torch.int32), "w": w * 2.5}
    sc = _score(l, s["score"])
    if op == "gate_grad":
        ids, dw = s["ids"].long(), s["dw"]
        c = sc.gather(1, ids)
        if s["renorm"]:
            total = c.sum(1, keepdim=True) + SUM_EPS
            dc = 2.5 * (dw - (dw * c).sum(1, keepdim=True) / total) / total
        else:
            dc = 2.5 * dw
        ds = torch.zeros_like(l).scatter_add_(1, ids, dc)
        if s["score"] == "softmax":
            dl = sc * (ds - (ds * sc).sum(1, keepdim=True))
        else:
            dl = ds * _score_slope(l, sc, s["score"])
        return dl if s["add"] is None else dl + s["add"]
    T, E = l.shape
    off = s["off"]
    if off is None:
        off = torch.tensor([0, T], dtype=torch.int32, device=l.device)
    B = off.numel() - 1
    t = torch.arange(T, device=l.device)
    seq = torch.searchsorted(off, t.to(torch.int32), right=True) - 1
    seq = torch.where(t < off[B], seq, B)                   # rows behind the last sequence: a bin that is dropped
    n = (off[1:] - off[:-1]).float()
    ids = s["ids"].long()
    counts = torch.zeros((B + 1) * (E + 1), dtype=torch.int32, device=l.device)
    at = seq[:, None] * (E + 1) + torch.where(ids >= 0, ids, E)
    counts.index_add_(0, at.reshape(-1), torch.ones(T * K, dtype=torch.int32, device=l.device))
    counts = counts.view(B + 1, E + 1)[:B, :E].contiguous()
    total = sc.sum(1, keepdim=True)
    p = sc / total
    inv = torch.where(n > 0, 1 / n, 0.0)
    f = counts.float() * (E / K) * inv[:, None]
    P = torch.zeros(B + 1, E, device=l.device).index_add_(0, seq, p)[:B] * inv[:, None]
    loss = 0.5 * (f * P).sum() / B
    a = torch.cat([f * (inv[:, None] * (0.5 / B)), torch.zeros(1, E, device=l.device)])[seq]
    a = a - (a * p).sum(1, keepdim=True)
    if s["score"] == "softmax":
        dl = p * a
    else:
        dl = a / total * _score_slope(l, sc, s["score"])
    return {"loss": loss.reshape(1), "counts": counts, "dlogits": dl}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        w = H * (4 if case["w32"] else 2)
        if op == "norm":
            return {"bytes": T * H * (2 + 2 + 1) + T * H // 128 + (4 * T * H if case["residual"] else 0) + w,
                    "flops": 8 * T * H}
        return {"bytes": T * H * (6 + (2 if case["dh"] else 0)) + w + 4 * H, "flops": 12 * T * H}
    if op in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * (4 if case["f32"] else 2)
        if op == "linear":
            return {"bytes": 2 * (M * K + N * K) + out * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
                    "flops": 2 * M * N * K}
        return {"bytes": 2 * (2 * M * K + 2 * N * K) + out + 4 * N + (4 * M * N if case["act"] != "none" else 0),
                "flops": 4 * M * N * K}
    T, E, K = case["T"], case["E"], case["K"]
    if op == "gate":
        return {"bytes": 4 * T * E + 8 * T * K + (4 * E if case["bias"] else 0), "flops": 10 * T * E}
    if op == "gate_grad":
        return {"bytes": 4 * T * E * (3 if case["add"] else 2) + 8 * T * K, "flops": 12 * T * E}
    return {"bytes": 8 * T * E + 4 * T * K + 4 * case["B"] * E, "flops": 16 * T * E}


# ------------------------------------------------------------------------------------------------- the exact outputs

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "norm":
        h = s["x"].to(d)
        if case["residual"]:
            h += s["res"].to(d)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["H"] + EPS) * s["w"].to(d)
        top = y.abs().view(case["T"], -1, 128).max(2).values
        e = torch.ceil(torch.log2(top / 448).clamp(min=-127))
        # a code's value before its rounding to 8 bits; a scale is a power of two, all or nothing
        return {"h": h, "y": y, "x_q": y / torch.exp2(e).repeat_interleave(128, 1), "x_s": None}
    if op == "norm_grad":
        h, dy, w = s["h"].to(d), s["dy"].to(d), s["w"].to(d)
        v = h.square().sum(1, keepdim=True) / case["H"] + EPS
        dot = (dy * w * h).sum(1, keepdim=True) / case["H"]
        dx = dy * w / v.sqrt() - h * dot / v.pow(1.5)
        if case["dh"]:
            dx += s["dh"].to(d)
        return {"dx": dx, "dw": (dy * h / v.sqrt()).sum(0)}
    if op in ("linear", "linear_grad"):
        def sigma(v):
            return 1 / (1 + torch.exp(-v))

        def cdf(v):
            return torch.special.ndtr(v)
        act = case["act"]
        if op == "linear":
            z = torch.matmul(s["x"].to(d), s["w"].to(d).t())
            z = z if s["b"] is None else z + s["b"].to(d)
            y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0), "silu": lambda: z * sigma(z),
                 "gelu": lambda: z * cdf(z), "sigmoid": lambda: sigma(z)}[act]()
            return y if s["res"] is None else y + s["res"].to(d)
        dz = s["dy"].to(d)
        if act != "none":
            z = s["z"].to(d)
            dz = dz * {"relu": lambda: torch.where(z > 0, 1.0, 0.0).to(d),
                       "silu": lambda: sigma(z) + z * sigma(z) * sigma(-z),
                       "gelu": lambda: cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi),
                       "sigmoid": lambda: sigma(z) * sigma(-z)}[act]()
        return {"dx": torch.matmul(dz, s["w"].to(d)), "dw": torch.matmul(dz.t(), s["x"].to(d)), "db": dz.sum(0)}
    l = s["logits"].to(d)
    dead = torch.isneginf(l)
    if case["score"] == "softmax":
        sc = torch.where(dead, 0.0, torch.exp(l - torch.where(dead, 0.0, torch.logsumexp(l, 1, keepdim=True))))
    elif case["score"] == "sigmoid":
        sc = 1 / (1 + torch.exp(-l))
    else:
        sc = torch.logaddexp(l, torch.zeros_like(l)).sqrt()
    T, E, K = case["T"], case["E"], case["K"]
    if op == "gate":
        key = l.clone() if s["bias"] is None else sc + s["bias"].to(d)
        key[dead] = -math.inf
        if case["pad"]:
            key[T - case["pad"]:] = -math.inf
        ids, w = [], []
        for _ in range(K):                                  # one pick after another; max over equal keys: the first
            best = key.max(1, keepdim=True).values
            first = (key == best).to(torch.int8).argmax(1, keepdim=True)
            none = torch.isneginf(best)
            ids.append(torch.where(none, -1, first))
            w.append(torch.where(none, 0.0, sc.gather(1, first)))
            key.scatter_(1, first, -math.inf)
        ids, w = torch.cat(ids, 1), torch.cat(w, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + SUM_EPS)
        return {"ids": ids.to(torch.int32), "w": 2.5 * w}
    hot = torch.zeros(T, E, dtype=d, device=l.device)
    if op == "gate_grad":
        chosen = hot.scatter(1, s["ids"].long(), 1.0)
        up = hot.scatter(1, s["ids"].long(), s["dw"].to(d)) * 2.5      # d loss / d weight, spread over the experts
        if case["renorm"]:
            total = (sc * chosen).sum(1, keepdim=True) + SUM_EPS
            up = (up - (up * sc).sum(1, keepdim=True) / total) * chosen / total
    else:
        off = [0, T] if s["off"] is None else s["off"].tolist()
        B = len(off) - 1
        total = sc.sum(1, keepdim=True)
        up, loss = hot, torch.zeros(1, dtype=d, device=l.device)
        counts = torch.zeros(B, E, dtype=torch.int32, device=l.device)
        for b in range(B):
            lo, hi = off[b], off[b + 1]
            if hi > lo:
                ids = s["ids"][lo:hi].long()
                counts[b] = torch.bincount(ids[ids >= 0], minlength=E).to(torch.int32)
                f = counts[b].to(d) * E / (K * (hi - lo))
                p = sc[lo:hi] / total[lo:hi]
                loss += 0.5 / B * (f * p.mean(0)).sum()
                up[lo:hi] = 0.5 / B / (hi - lo) * (f - (p * f).sum(1, keepdim=True)) / total[lo:hi]
    if case["score"] == "softmax":
        dl = sc * up - sc * (sc * up).sum(1, keepdim=True)
    elif case["score"] == "sigmoid":
        dl = up * sc * (1 - sc)
    else:
        dl = up * (1 / (1 + torch.exp(-l))) / (2 * sc)
    if op == "gate_grad":
        return dl if s["add"] is None else dl + s["add"].to(d)
    return {"loss": loss, "counts": counts, "dlogits": dl}
