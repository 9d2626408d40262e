"""Operators between a private language model's linears, as a user's program calls them.

Each case names one pass through one operator: attention over the batch's sequences
(causal or not, grouped heads, several documents in a row, padding) and its gradients,
the norms of queries and keys with the rotation by their positions and the gradients
of both (the norm weights' per sample, for clipping), and dropout whose mask is drawn
from a counter and never stored.  With ``own`` false ``run`` computes the pass from
elementary torch operations in float32; with ``own`` true it calls this repository's
package.  ``exact`` gives the definition's values in float64.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BASE = 10000.0

# The largest listed sizes: drawn cases cost no more than these.
MOST_SCORES = 8 * 40 * 2048 * 2048 * 128   # batch x heads x queries x keys x head width
MOST_HEADS = 8 * 2048 * 80 * 128           # entries of queries and keys together
MOST_ENTRIES = 8 * 2048 * 5120             # entries that dropout passes over


def _attn(name, op, B, T, Hq, Hkv, D, dtype, Tk=None, causal=True, masked=False, docs=0, fused=False):
    return {"name": name, "op": op, "B": B, "T": T, "Tk": T if Tk is None else Tk, "Hq": Hq,
            "Hkv": Hkv, "D": D, "dtype": dtype, "causal": causal, "masked": masked, "docs": docs,
            "fused": fused}


def _rot(name, op, B, T, Hq, Hkv, D, dtype, rot, norm=True, interleaved=False, masked=False,
         far=0, restart=False):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "rot": rot, "norm": norm, "interleaved": interleaved, "masked": masked, "far": far,
            "restart": restart}


def listed():
    return [
        # the next token of sixteen sequences over the positions before it: bytes of the keys and values
        _attn("attention 16x1 over 4096, 40/8x128", "attn", 16, 1, 40, 8, 128, "bf16", Tk=4096),
        # a ragged batch of a RoBERTa-large-sized encoder, queries, keys and values of one product
        _attn("attention 32x128, 16x64, both ways, ragged", "attn", 32, 128, 16, 16, 64, "bf16",
              causal=False, masked=True, fused=True),
        # a Llama-13B layer's batch
        _attn("attention 8x2048, 40x128", "attn", 8, 2048, 40, 40, 128, "bf16"),
        # documents of different lengths packed into one row, grouped heads
        _attn("attention 1x8192 packed, 40/8x128", "attn", 1, 8192, 40, 8, 128, "bf16", docs=6),
        # a small odd model in float32, ragged: latency and element-wise loads
        _attn("attention_bwd 3x77, 6/2x45, ragged", "attn_bwd", 3, 77, 6, 2, 45, "f32", masked=True),
        # a GPT-2-small layer's batch
        _attn("attention_bwd 32x512, 12x64", "attn_bwd", 32, 512, 12, 12, 64, "bf16", fused=True),
        # a Llama-13B layer's batch
        _attn("attention_bwd 8x2048, 40x128", "attn_bwd", 8, 2048, 40, 40, 128, "bf16"),
        # the next token of sixteen sequences far into their contexts: latency
        _rot("rotary 16x1, 40/8x128", "rotary", 16, 1, 40, 8, 128, "bf16", 128, far=100000),
        # a Llama-13B layer's batch
        _rot("rotary 8x2048, 40x128", "rotary", 8, 2048, 40, 40, 128, "bf16", 128),
        # its gradients, packed documents, half of each head rotated
        _rot("rotary_bwd 8x2048, 40x128", "rotary_bwd", 8, 2048, 40, 40, 128, "bf16", 64,
             interleaved=True, restart=True),
        # a small odd model in float32, ragged: latency and element-wise loads
        {"name": "dropout 4x33x99", "op": "dropout", "B": 4, "T": 33, "D": 99, "dtype": "f32",
         "p": 0.1, "residual": False, "masked": True},
        # the branch of a Llama-13B layer added to its stream
        {"name": "dropout 8x2048x5120", "op": "dropout", "B": 8, "T": 2048, "D": 5120,
         "dtype": "bf16", "p": 0.1, "residual": True, "masked": False},
    ]


def _logint(rng, lo, hi):
    """An integer whose logarithm is uniform over the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_bwd", "attn_bwd", "rotary", "rotary_bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    B, T = _logint(rng, 1, 32), _logint(rng, 1, 4096)
    masked = rng.random() < 0.4
    if op == "dropout":
        D = _logint(rng, 16, 5120)
        return {"op": op, "B": B, "T": max(1, min(T, MOST_ENTRIES // (2 * B * D))), "D": D,
                "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.3, 0.5]),
                "residual": rng.random() < 0.5, "masked": masked}
    Hkv, group = _logint(rng, 1, 16), rng.choice([1, 1, 2, 4, 5, 8])
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, rng.randint(8, 128), 2 * rng.randint(4, 64)])
    if op in ("rotary", "rotary_bwd"):
        D += D % 2
        T = max(1, min(T, MOST_HEADS // (2 * B * Hkv * (group + 1) * D)))
        c = _rot("", op, B, T, Hkv * group, Hkv, D, dtype, rng.choice([D, D, 2 * max(1, D // 4)]),
                 norm=rng.random() < 0.7, interleaved=rng.random() < 0.4, masked=masked,
                 far=rng.choice([0, 0, 30000, 1000000]), restart=rng.random() < 0.3)
    else:
        # float32 matrix products run at a tenth of the rate
        room = MOST_SCORES // (10 if dtype == "f32" else 1) // (B * Hkv * group * D)
        T = max(1, min(T, int(math.isqrt(room))))
        c = _attn("", op, B, T, Hkv * group, Hkv, D, dtype, causal=rng.random() < 0.75, masked=masked,
                  docs=rng.choice([0, 0, 0, _logint(rng, 2, 12)]) if T >= 16 else 0,
                  fused=rng.random() < 0.4)
        if op == "attn" and rng.random() < 0.35:
            # a few new tokens over those before them
            c["T"] = _logint(rng, 1, 64)
            c["Tk"] = max(c["T"], min(_logint(rng, 64, 8192), room // c["T"],
                                      (1 << 27) // (B * Hkv * D)))
            c["docs"], c["fused"] = 0, False
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths_mask(g, B, T, front=False):
    """Padding at the end (or in front): sample i keeps T_i tokens, T/16 <= T_i <= T."""
    n = torch.randint(max(1, T // 16), T + 1, (B, 1), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")[None, :]
    return ((t >= T - n) if front else (t < n)).to(torch.uint8)


def _documents(g, B, T, docs):
    """Non-decreasing document numbers of a row's tokens: its cuts are random."""
    cuts = torch.randint(1, max(2, T), (B, docs - 1), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    return (t[None, :, None] >= cuts[:, None, :]).sum(-1).to(torch.int32)


def _randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)


def _heads(g, c, dt, T, Tk):
    """q, k, v: tensors of their own, or the parts of one product's rows."""
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    if c.get("fused"):
        rows = _randn(g, (B, T, (Hq + 2 * Hkv) * D), dt, 1.3)
        q, k, v = rows.split([Hq * D, Hkv * D, Hkv * D], dim=2)
        return q.unflatten(2, (Hq, D)), k.unflatten(2, (Hkv, D)), v.unflatten(2, (Hkv, D))
    return (_randn(g, (B, T, Hq, D), dt, 1.3), _randn(g, (B, Tk, Hkv, D), dt, 1.3),
            _randn(g, (B, Tk, Hkv, D), dt))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B, T, dt = case["op"], case["B"], case["T"], _DT[case["dtype"]]
    s = {"case": case, "op": op, "mask": None}
    if op == "dropout":
        s["x"] = _randn(g, (B, T, case["D"]), dt)
        s["residual"] = _randn(g, (B, T, case["D"]), dt, 3.0) if case["residual"] else None
        s["mask"] = _lengths_mask(g, B, T) if case["masked"] else None
        s["seed"], s["offset"] = int(seed) * 0x9E3779B97F4A7C15 % (1 << 63), 11
        return s
    if op in ("attn", "attn_bwd"):
        Tk = case["Tk"]
        s["q"], s["k"], s["v"] = _heads(g, case, dt, T, Tk)
        if case["masked"]:
            s["mask"] = _lengths_mask(g, B, Tk, front=Tk != T)
        s["segments"] = _documents(g, B, Tk, case["docs"]) if case["docs"] else None
        if op == "attn_bwd":
            s["out"], s["lse"] = _plain_attn(s, case)    # what the forward pass kept
            s["dout"] = _randn(g, s["q"].shape, dt, 1e-2)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    s["q"], s["k"] = _randn(g, (B, T, Hq, D), dt, 2.0), _randn(g, (B, T, Hkv, D), dt, 2.0)
    s["wq"] = 1.0 + _randn(g, (D,), torch.float32, 0.1) if case["norm"] else None
    s["wk"] = 1.0 + _randn(g, (D,), torch.float32, 0.1) if case["norm"] else None
    # the rotation of pair j by one position, in radians
    s["freqs"] = BASE ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    s["positions"] = None
    if case["far"] or case["restart"]:
        t = torch.arange(T, device="cuda")[None, :].expand(B, T)
        if case["restart"]:
            doc = _documents(g, B, T, 4)
            first = torch.searchsorted(doc, doc)
            t = t - first
        if case["far"]:
            t = t + torch.randint(0, case["far"], (B, 1), generator=g, device="cuda")
        s["positions"] = t.contiguous()
    s["mask"] = _lengths_mask(g, B, T) if case["masked"] else None
    if op == "rotary_bwd":
        s["dq"], s["dk"] = _randn(g, s["q"].shape, dt, 1e-2), _randn(g, s["k"].shape, dt, 1e-2)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _chunks(c):
    """Samples and key heads whose scores are formed together: at most 2^29 of them."""
    B, Hkv, per = c["B"], c["Hkv"], c["Hq"] // c["Hkv"] * c["T"] * c["Tk"]
    heads = max(1, min(Hkv, (1 << 29) // per))
    rows = max(1, (1 << 29) // (per * Hkv)) if heads == Hkv else 1
    return [(slice(b, min(b + rows, B)), slice(h, min(h + heads, Hkv)))
            for b in range(0, B, rows) for h in range(0, Hkv, heads)]


def _allowed(s, c, b):
    """[samples, 1, 1, T, Tk] truth values: the query attends to the key."""
    T, Tk = c["T"], c["Tk"]
    key = torch.arange(Tk, device="cuda")
    ok = torch.ones((1, T, Tk), dtype=torch.bool, device="cuda")
    if c["causal"]:
        ok = ok & (key[None, None, :] <= key[Tk - T:][None, :, None])
    if s["segments"] is not None:
        seg = s["segments"][b]
        ok = ok & (seg[:, Tk - T:, None] == seg[:, None, :])
    if s["mask"] is not None:
        m = s["mask"][b] != 0
        ok = ok & m[:, Tk - T:, None] & m[:, None, :]
    return ok[:, None, None]


def _grouped(x, b, h, heads):
    """x [B, T, heads * g, D] -> float32 [samples, key heads, g, T, D]."""
    x = x[b].float()
    return x.unflatten(2, (heads, -1))[:, :, h].permute(0, 2, 3, 1, 4).contiguous()


def _scores(s, c, b, h):
    q, k = _grouped(s["q"], b, h, c["Hkv"]), _grouped(s["k"], b, h, c["Hkv"])
    n, H, G, T, D = q.shape
    S = torch.matmul(q.reshape(n, H, G * T, D), k[:, :, 0].transpose(-1, -2).contiguous())
    S = (S * (1.0 / math.sqrt(D))).reshape(n, H, G, T, -1)
    return q, k[:, :, 0], S.masked_fill(~_allowed(s, c, b), float("-inf"))


def _plain_attn(s, c):
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    lse = torch.empty((c["B"], c["Hq"], c["T"]), device="cuda")
    by_head = out.unflatten(2, (c["Hkv"], -1))
    for b, h in _chunks(c):
        _, _, S = _scores(s, c, b, h)
        m = S.amax(-1, keepdim=True)
        m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
        P = torch.exp(S - m)
        total = P.sum(-1, keepdim=True)
        empty = total == 0
        v = _grouped(s["v"], b, h, c["Hkv"])[:, :, 0]
        O = torch.matmul(P.flatten(2, 3), v).reshape(*P.shape[:4], -1)
        O = torch.where(empty, torch.zeros_like(O), O / total)
        by_head[b, :, h] = O.permute(0, 3, 1, 2, 4).to(out.dtype)
        L = torch.where(empty, torch.zeros_like(m), m + torch.log(total))[..., 0]
        lse.unflatten(1, (c["Hkv"], -1))[b, h] = L
    return out, lse


def _plain_attn_bwd(s, c):
    grads = [torch.empty(s[x].shape, dtype=s[x].dtype, device="cuda") for x in "qkv"]
    dq, dk, dv = (x.unflatten(2, (c["Hkv"], -1)) for x in grads)
    for b, h in _chunks(c):
        q, k, S = _scores(s, c, b, h)
        L = s["lse"].unflatten(1, (c["Hkv"], -1))[b, h]
        P = torch.exp(S - L[..., None])
        del S
        v, do = _grouped(s["v"], b, h, c["Hkv"])[:, :, 0], _grouped(s["dout"], b, h, c["Hkv"])
        n, H, G, T, D = q.shape
        flat = P.reshape(n, H, G * T, -1)
        dv[b, :, h, 0] = torch.matmul(flat.transpose(-1, -2).contiguous(),
                                      do.reshape(n, H, G * T, D)).transpose(1, 2).to(dv.dtype)
        dP = torch.matmul(do.reshape(n, H, G * T, D), v.transpose(-1, -2).contiguous()).reshape(P.shape)
        dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * (1.0 / math.sqrt(D))
        del P, dP, flat
        dS = dS.reshape(n, H, G * T, -1)
        dq[b, :, h] = torch.matmul(dS, k).reshape(n, H, G, T, D).permute(0, 3, 1, 2, 4).to(dq.dtype)
        dk[b, :, h, 0] = torch.matmul(dS.transpose(-1, -2).contiguous(),
                                      q.reshape(n, H, G * T, D)).transpose(1, 2).to(dk.dtype)
    return grads


def _angles(s, c):
    """cos and sin [B or 1, T, 1, pairs]; the angles of far positions need float64."""
    at = torch.arange(c["T"], device="cuda")[None] if s["positions"] is None else s["positions"]
    a = at.double()[:, :, None, None] * s["freqs"]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin, c):
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _kept(s, x):
    return x if s["mask"] is None else x * (s["mask"] != 0)[:, :, None, None]


def _plain_rotary(s, c):
    cos, sin = _angles(s, c)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
        out.append(_kept(s, _turn(y, cos, sin, c)).to(x.dtype))
    return out


def _plain_rotary_bwd(s, c):
    cos, sin = _angles(s, c)
    grads, weights = [], []
    for x, dy, w in ((s["q"], s["dq"], s["wq"]), (s["k"], s["dk"], s["wk"])):
        d = _kept(s, _turn(dy.float(), cos, -sin, c))
        if w is not None:
            y = x.float()
            r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
            y = y * r
            weights.append((d * y).sum((1, 2))[:, None])
            d = d * w
            d = r * (d - y * (d * y).mean(-1, keepdim=True))
        grads.append(d.to(x.dtype))
    return grads + weights


_M32 = 0xFFFFFFFF


def _plain_dropout(s, c):
    """Entry e is kept where the 16-bit half e mod 8 of Philox block offset + e / 8, counter
    (low, high, 1, 0), is at least 65536 p."""
    n = s["x"].numel()
    j = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64) + s["offset"]
    w = [j & _M32, (j >> 32) & _M32, torch.ones_like(j), torch.zeros_like(j)]
    k0, k1 = s["seed"] & _M32, s["seed"] >> 32
    for r in range(10):
        p0, p1 = w[0] * 0xD2511F53, w[2] * 0xCD9E8D57
        w = [((p1 >> 32) & _M32) ^ w[1] ^ k0, p1 & _M32, ((p0 >> 32) & _M32) ^ w[3] ^ k1, p0 & _M32]
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    halves = torch.stack([h for x in w for h in (x & 0xFFFF, x >> 16)], 1).reshape(-1)[:n]
    limit = round(c["p"] * 65536)
    y = s["x"].float() * (65536.0 / (65536 - limit))
    y = torch.where((halves >= limit).view_as(y), y, torch.zeros_like(y))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if s["mask"] is not None:
        y = y * (s["mask"] != 0)[:, :, None]
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------------------
def run(state):
    c, op = state["case"], state["op"]
    if not own:
        return {"attn": _plain_attn, "attn_bwd": _plain_attn_bwd, "rotary": _plain_rotary,
                "rotary_bwd": _plain_rotary_bwd, "dropout": _plain_dropout}[op](state, c)
    import sample_gradient_clipping_amd as dp
    if op == "attn":
        r = dp.attention(state["q"], state["k"], state["v"], mask=state["mask"],
                         segments=state["segments"], causal=c["causal"])
        return r.out, r.lse
    if op == "attn_bwd":
        return dp.attention_backward(state["dout"], state["q"], state["k"], state["v"], state["out"],
                                     state["lse"], mask=state["mask"], segments=state["segments"],
                                     causal=c["causal"])
    if op == "rotary":
        return dp.qk_norm_rotary(state["q"], state["k"], state["wq"], state["wk"],
                                 freqs=state["freqs"], positions=state["positions"],
                                 mask=state["mask"], interleaved=c["interleaved"], eps=EPS)
    if op == "rotary_bwd":
        r = dp.qk_norm_rotary_backward(state["dq"], state["dk"], state["q"], state["k"], state["wq"],
                                       state["wk"], freqs=state["freqs"],
                                       positions=state["positions"], mask=state["mask"],
                                       interleaved=c["interleaved"], eps=EPS)
        return [x for x in r if x is not None]
    return dp.dropout(state["x"], c["p"], seed=state["seed"], offset=state["offset"],
                      residual=state["residual"], mask=state["mask"])


# ---------------------------------------------------------------------------
def _pairs(c):
    """Expected number of (query, key) pairs of a head over the batch."""
    B, T, Tk = c["B"], c["T"], c["Tk"]
    if T != Tk:
        each = (T * (Tk - T) + T * (T + 1) / 2) if c["causal"] else T * Tk
        return B * each * (0.53 if c["masked"] else 1.0)
    square = float(T * T)
    if c["masked"]:
        square *= 0.355       # lengths uniform over (T/16, T)
    if c["docs"]:
        square *= 2.0 / (c["docs"] + 1)
    return B * (square / 2 + T / 2 if c["causal"] else square)


def work(case):
    """Bytes and operations a pass cannot do without: inputs read once, outputs written once."""
    op, N = case["op"], case["B"] * case["T"]
    b = {"bf16": 2, "f32": 4}[case["dtype"]]
    kept = 0.53 if case["masked"] else 1.0
    if op == "dropout":
        n = N * case["D"]
        return {"bytes": n * b * (kept * (2 if case["residual"] else 1) + 1), "flops": 2 * kept * n}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op in ("rotary", "rotary_bwd"):
        n = N * (Hq + Hkv) * D
        reads = 1 if op == "rotary" or not case["norm"] else 2
        flops = (6 if case["norm"] else 3) * (1 if op == "rotary" else 2)
        return {"bytes": n * b * (kept * reads + 1), "flops": kept * flops * n}
    keys = case["B"] * case["Tk"] * Hkv * D
    if op == "attn":
        return {"bytes": b * ((1 + kept) * N * Hq * D + 2 * kept * keys) + 4 * N * Hq,
                "flops": 4 * D * Hq * _pairs(case)}
    return {"bytes": b * ((3 * kept + 1) * N * Hq * D + (2 * kept + 2) * keys) + 4 * kept * N * Hq,
            "flops": 10 * D * Hq * _pairs(case)}


# ---------------------------------------------------------------------------
# The definitions in float64
# ---------------------------------------------------------------------------
def _exact_attn(s, c):
    """Head by head: softmax over the keys a query may see, gradients by automatic differentiation."""
    B, T, Tk, Hq, Hkv = c["B"], c["T"], c["Tk"], c["Hq"], c["Hkv"]
    back = c["op"] == "attn_bwd"
    outs, lses = [], []
    grads = [torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"] if back else None
    at = torch.arange(Tk, device="cuda")
    for b in range(B):
        here = torch.ones(Tk, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][b] != 0
        doc = torch.zeros_like(at) if s["segments"] is None else s["segments"][b]
        hide = (doc[Tk - T:, None] != doc[None, :]) | ~here[None, :]
        if c["causal"]:
            hide |= at[None, :] > at[Tk - T:, None]
        live = here[Tk - T:]
        hide[~live] = False          # those queries are set to zero below
        for h in range(Hq):
            q, k, v = (s[x][b, :, y].double().requires_grad_(back)
                       for x, y in (("q", h), ("k", h * Hkv // Hq), ("v", h * Hkv // Hq)))
            z = (q @ k.T / math.sqrt(c["D"])).masked_fill(hide, float("-inf"))
            o = (torch.softmax(z, -1) @ v) * live[:, None]
            if back:
                # masked queries' outputs are zero whatever came in for them
                for x, d, y in zip(grads, torch.autograd.grad(o, (q, k, v), s["dout"][b, :, h].double()),
                                   (h, h * Hkv // Hq, h * Hkv // Hq)):
                    x[b, :, y] += d
            else:
                outs.append(o)
                lses.append(torch.where(live, torch.logsumexp(z, -1), 0.0))
    if back:
        return grads
    out = torch.stack(outs).reshape(B, Hq, T, -1).transpose(1, 2)
    return out, torch.stack(lses).reshape(B, Hq, T)


def _exact_rotary(s, c):
    """The rotation as a complex product, the norm's gradients by automatic differentiation."""
    B, T, half = c["B"], c["T"], c["rot"] // 2
    at = torch.arange(T, device="cuda").expand(B, T) if s["positions"] is None else s["positions"]
    unit = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       at.double()[..., None] * s["freqs"])
    live = torch.ones((B, T), device="cuda") if s["mask"] is None else (s["mask"] != 0)
    values, grads, weights = [], [], []
    for x, w, d in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        parts, dparts, wparts = [], [], []
        for b in range(B):
            y = x[b].double().requires_grad_(d is not None)
            n, wb = y, None
            if w is not None:
                wb = w.double().clone().requires_grad_(d is not None)
                n = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * wb
            head, rest = n[..., : 2 * half], n[..., 2 * half:]
            pairs = head.unflatten(-1, (half, 2)) if c["interleaved"] else \
                head.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit[b][:, None, :])
            z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            z = torch.cat([z, rest], -1) * live[b][:, None, None]
            if d is None:
                parts.append(z)
                continue
            got = torch.autograd.grad(z, (y,) if wb is None else (y, wb), d[b].double())
            dparts.append(got[0])
            if wb is not None:
                wparts.append(got[1][None])
        if d is None:
            values.append(torch.stack(parts))
        else:
            grads.append(torch.stack(dparts))
            weights += [torch.stack(wparts)] if wparts else []
    return values + grads + weights


def _exact_dropout(s, c):
    x = s["x"].double().cpu().numpy().reshape(-1)
    n, lim = x.size, round(c["p"] * 65536)
    keep = np.empty((n + 7) // 8 * 8, dtype=bool)
    step = 1 << 20
    for a in range(0, keep.size // 8, step):
        j = np.arange(a, min(a + step, keep.size // 8), dtype=np.uint64) + np.uint64(s["offset"])
        c0, c1 = j.astype(np.uint32), (j >> np.uint64(32)).astype(np.uint32)
        c2, c3 = np.ones_like(c0), np.zeros_like(c0)
        for r in range(10):
            k0 = np.uint32((s["seed"] + r * 0x9E3779B9) % 2 ** 32)
            k1 = np.uint32((s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32)
            a0 = c0.astype(np.uint64) * np.uint64(0xD2511F53)
            a1 = c2.astype(np.uint64) * np.uint64(0xCD9E8D57)
            c0, c1 = (a1 >> np.uint64(32)).astype(np.uint32) ^ c1 ^ k0, a1.astype(np.uint32)
            c2, c3 = (a0 >> np.uint64(32)).astype(np.uint32) ^ c3 ^ k1, a0.astype(np.uint32)
        words = np.stack([c0, c1, c2, c3], 1).astype("<u4").view("<u2")
        keep[8 * a: 8 * a + words.size] = words.reshape(-1) >= lim
    y = np.where(keep[:n], x * 65536.0 / (65536 - lim), 0.0).reshape(tuple(s["x"].shape))
    y = torch.from_numpy(y).cuda()
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return y if s["mask"] is None else torch.where((s["mask"] != 0)[..., None], y, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn", "attn_bwd"):
        return _exact_attn(s, case)
    return _exact_dropout(s, case) if op == "dropout" else _exact_rotary(s, case)
