"""Operators of a private language-model step, as a user's program calls them.

Each case names one pass through one operator: the embedding lookup, the
embedding's per-sample clipped gradient, the log probabilities of given tokens,
their gradient to the logits, and the orthogonalised update (alone, or as a whole
optimizer step).  With ``own`` false ``run`` computes the pass from elementary
torch operations in float32; with ``own`` true it calls this repository's package.
``exact`` gives the definition's values in float64.
"""
import math

import numpy as np
import torch

own = False

NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7

# The largest listed sizes: drawn cases cost no more than these.
MOST_ROWS = 8 * 2048            # tokens of a batch
MOST_WIDTH = 5120               # model width
MOST_TABLE = 32000 * 5120       # entries of an embedding table
MOST_LOGITS = 8 * 2048 * 32000  # logits of a batch


def listed():
    return [
        # sixteen sequences' next token from a float32 master table: latency
        {"name": "lookup 16x1 50257x768", "op": "lookup", "B": 16, "T": 1, "V": 50257, "D": 768,
         "dtype": "f32", "out": "bf16", "ids": "i64", "masked": False, "scale": 1.0},
        # a training batch of the Llama-13B width, rows scaled on the way
        {"name": "lookup 8x2048 32000x5120", "op": "lookup", "B": 8, "T": 2048, "V": 32000, "D": 5120,
         "dtype": "bf16", "out": "bf16", "ids": "i64", "masked": False, "scale": 71.55},
        # a small odd model in float32, ragged: latency and element-wise loads
        {"name": "embgrad 4x33 1001x99", "op": "embgrad", "B": 4, "T": 33, "V": 1001, "D": 99,
         "dtype": "f32", "ids": "i32", "masked": True, "scale": 2.0, "sigma": 0.0, "accumulate": False},
        # the whole private gradient of a GPT-2-small table, noise included
        {"name": "embgrad 32x512 50257x768", "op": "embgrad", "B": 32, "T": 512, "V": 50257, "D": 768,
         "dtype": "bf16", "ids": "i64", "masked": False, "scale": 1.0, "sigma": 0.8, "accumulate": False},
        # one ragged micro-batch of a Llama-13B-wide table, added to earlier ones
        {"name": "embgrad 8x2048 32000x5120", "op": "embgrad", "B": 8, "T": 2048, "V": 32000, "D": 5120,
         "dtype": "bf16", "ids": "i64", "masked": True, "scale": 1.0, "sigma": 0.0, "accumulate": True},
        # one decoded token with its five best alternatives: latency
        {"name": "logprobs 1x1 32000 top5", "op": "logprobs", "B": 1, "T": 1, "V": 32000,
         "dtype": "bf16", "ids": "i64", "masked": False, "top_k": 5},
        # scoring a ragged batch: rows of odd length, alternatives wanted
        {"name": "logprobs 4x513 50257 top8", "op": "logprobs", "B": 4, "T": 513, "V": 50257,
         "dtype": "f32", "ids": "i32", "masked": True, "top_k": 8},
        # the loss of a training batch
        {"name": "logprobs 8x2048 32000", "op": "logprobs", "B": 8, "T": 2048, "V": 32000,
         "dtype": "bf16", "ids": "i64", "masked": False, "top_k": 0},
        # its gradient, rows of odd length, with an entropy term
        {"name": "logprobs_bwd 4x513 50257", "op": "logprobs_bwd", "B": 4, "T": 513, "V": 50257,
         "dtype": "f32", "ids": "i32", "masked": True, "entropy": True},
        # the gradient of the training batch: the head linear's G
        {"name": "logprobs_bwd 8x2048 32000", "op": "logprobs_bwd", "B": 8, "T": 2048, "V": 32000,
         "dtype": "bf16", "ids": "i64", "masked": False, "entropy": False},
        # the attention projections of three GPT-2-small layers orthogonalised together
        {"name": "ortho 12x768x768", "op": "ortho", "n": 12, "dout": 768, "din": 768,
         "dtype": "bf16", "steps": 5},
        # the optimizer step of one Llama-13B MLP matrix
        {"name": "muon 13824x5120", "op": "muon", "n": 1, "dout": 13824, "din": 5120,
         "dtype": "f32", "steps": 5},
    ]


def _logint(rng, lo, hi):
    """An integer whose logarithm is uniform over the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "embgrad", "embgrad", "logprobs", "logprobs", "logprobs_bwd", "ortho", "muon"])
    dt = rng.choice(["bf16", "f32"])
    if op in ("ortho", "muon"):
        dout, din = _logint(rng, 16, 6000), _logint(rng, 16, 6000)
        n = max(1, min(_logint(rng, 1, 16), (5120 * 5120) // (dout * din)))
        return {"op": op, "n": n, "dout": dout, "din": din, "dtype": dt if op == "ortho" else "f32",
                "steps": rng.choice([3, 5, 6])}
    B = _logint(rng, 1, 64)
    T = max(1, min(_logint(rng, 1, 4096), MOST_ROWS // B))
    case = {"op": op, "B": B, "T": T, "dtype": dt, "ids": rng.choice(["i32", "i64"]),
            "masked": rng.random() < 0.5}
    if op in ("lookup", "embgrad"):
        D = _logint(rng, 32, MOST_WIDTH)
        V = max(2, min(_logint(rng, 256, 131072), MOST_TABLE // D))
        if dt == "f32":
            V = max(2, min(V, MOST_TABLE // (2 * D)))
        if rng.random() < 0.5:
            D = max(8, D // 8 * 8)
        case.update(V=V, D=D, scale=rng.choice([1.0, 27.5]))
        if op == "lookup":
            case.update(out=rng.choice(["bf16", "f32"]))
        else:
            case.update(sigma=rng.choice([0.0, 0.8]), accumulate=rng.random() < 0.5)
        return case
    V = _logint(rng, 256, 262144)
    if rng.random() < 0.5:
        V = max(8, V // 8 * 8)
    room = MOST_LOGITS // (2 if dt == "f32" else 1)
    case["T"] = max(1, min(case["T"], room // (B * V)))
    case["V"] = V
    if op == "logprobs":
        case.update(top_k=rng.choice([0, 1, 5, 8]))
    else:
        case.update(entropy=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_IT = {"i32": torch.int32, "i64": torch.int64}
_M32 = 0xFFFFFFFF


def _philox_normals(seed, offset, n):
    """xi_e, e < n: the Philox4x32-10 / Box-Muller law of the library's noise, in float64."""
    blocks = (n + 3) // 4
    j = torch.arange(blocks, device="cuda", dtype=torch.int64) + offset
    c = [j & _M32, (j >> 32) & _M32, torch.zeros_like(j), torch.zeros_like(j)]
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for r in range(10):
        if r:
            k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & _M32) ^ c[1] ^ k0, p1 & _M32, ((p0 >> 32) & _M32) ^ c[3] ^ k1, p0 & _M32]
    u = [((w >> 9).double() + 0.5) * 2.0 ** -23 for w in c]
    ra, rb = torch.sqrt(-2 * torch.log(u[0])), torch.sqrt(-2 * torch.log(u[2]))
    ta, tb = 2 * math.pi * u[1], 2 * math.pi * u[3]
    z = torch.stack([ra * torch.cos(ta), ra * torch.sin(ta), rb * torch.cos(tb), rb * torch.sin(tb)], 1)
    return z.reshape(-1)[:n]


def _tokens(g, B, T, V, dt):
    """Token ids whose frequencies fall with their rank (log-uniform ranks), in a shuffled vocabulary."""
    u = torch.rand((B, T), generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    return torch.randperm(V, generator=g, device="cuda")[rank].to(dt)


def _mask(g, B, T):
    """Padding at the end: sample i keeps its first T_i tokens, 1 <= T_i <= T (T/16 at least)."""
    lo = max(1, T // 16)
    lengths = torch.randint(lo, T + 1, (B,), generator=g, device="cuda")
    return (torch.arange(T, device="cuda")[None, :] < lengths[:, None]).to(torch.uint8)


def _randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("ortho", "muon"):
        shape = (case["n"], case["dout"], case["din"]) if case["n"] > 1 else (case["dout"], case["din"])
        dt = _DT[case["dtype"]]
        # a privatised gradient: a low-rank part under Gaussian noise
        k = min(8, case["dout"], case["din"])
        left = torch.randn(shape[:-1] + (k,), generator=g, device="cuda")
        right = torch.randn(shape[:-2] + (k, shape[-1]), generator=g, device="cuda")
        s["grad"] = ((torch.matmul(left, right) / math.sqrt(k)
                      + torch.randn(shape, generator=g, device="cuda")) * 1e-3).to(dt)
        if op == "muon":
            s["momentum"] = _randn(g, shape, torch.float32, 3e-3)
            s["W"] = _randn(g, shape, torch.float32, 0.02)
        return s
    B, T, V = case["B"], case["T"], case["V"]
    dt = _DT[case["dtype"]]
    s["ids"] = _tokens(g, B, T, V, _IT[case["ids"]])
    s["mask"] = _mask(g, B, T) if case["masked"] else None
    if op == "lookup":
        s["table"] = _randn(g, (V, case["D"]), dt, 0.02)
    elif op == "embgrad":
        D = case["D"]
        per_sample = torch.exp(torch.randn((B, 1, 1), generator=g, device="cuda"))
        s["G"] = (torch.randn((B, T, D), generator=g, device="cuda") * per_sample * 1e-3).to(dt)
        # a clip norm in the middle of the samples' norms: about half are clipped
        s["C"] = 1e-3 * math.sqrt(T * D) * case["scale"]
        s["denom"] = float(2 * B) if case["accumulate"] else float(B)
        s["noise"] = int(seed)
        if case["accumulate"]:
            s["grad"] = _randn(g, (V, D), torch.float32, 1e-4)
        if case["sigma"] > 0:
            s["xi"] = _philox_normals(int(seed), 7, V * D).float().reshape(V, D)
    else:
        s["logits"] = _randn(g, (B, T, V), dt, 2.5)
        # a trained model gives its target more than chance
        at = s["ids"].long().unsqueeze(-1)
        s["logits"].scatter_add_(2, at, torch.full_like(at, 6, dtype=dt))
        if op == "logprobs_bwd":
            s["dlogp"] = _randn(g, (B, T), torch.float32, 0.1) - 1.0
            s["dentropy"] = _randn(g, (B, T), torch.float32, 0.1) if case["entropy"] else None
            z = s["logits"]
            lse, ent = torch.empty((B, T), device="cuda"), torch.empty((B, T), device="cuda")
            for b in range(B):  # what the forward pass kept
                w = z[b].float()
                lse[b] = torch.logsumexp(w, -1)
                ent[b] = lse[b] - (torch.exp(w - lse[b][:, None]) * w).sum(-1)
            s["lse"], s["entropy"] = lse, ent
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _active(s):
    m = s["mask"]
    return torch.ones_like(s["ids"], dtype=torch.bool) if m is None else m != 0


def _plain_lookup(s, c):
    rows = s["table"][s["ids"].long()].float() * c["scale"]
    return (rows * _active(s)[..., None]).to(_DT[c["out"]])


def _plain_embgrad(s, c):
    B, T, V, D = c["B"], c["T"], c["V"], c["D"]
    ids, act = s["ids"].long(), _active(s)
    # runs of one token within one sample, by sorting (sample, token)
    sample = torch.arange(B, device="cuda")[:, None].expand(B, T)
    key, order = torch.sort((sample * V + ids).reshape(-1))
    run = torch.cumsum(torch.cat([key.new_zeros(1), (key[1:] != key[:-1]).long()]), 0)
    rows = (s["G"].float() * act[..., None] * c["scale"]).reshape(B * T, D)[order]
    sums = torch.zeros((B * T, D), device="cuda").index_add_(0, run, rows)
    of_run = torch.zeros(B * T, dtype=torch.int64, device="cuda").scatter_(0, run, key)
    sq = torch.zeros(B, device="cuda").index_add_(0, of_run // V, (sums * sums).sum(1))
    norms = torch.sqrt(sq)
    factor = torch.where(norms <= s["C"], torch.ones_like(norms), s["C"] / norms)
    grad = torch.zeros((V, D), device="cuda").index_add_(0, of_run % V, sums * factor[of_run // V][:, None])
    if c["sigma"] > 0:
        grad = grad + (c["sigma"] * s["C"]) * s["xi"]
    grad = grad / s["denom"]
    if c["accumulate"]:
        s["grad"].add_(grad)
        grad = s["grad"]
    return grad, norms


def _plain_logprobs(s, c):
    z, act = s["logits"].float(), _active(s)
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1)
    lse = m.squeeze(-1) + torch.log(total)
    entropy = torch.log(total) - (e * d).sum(-1) / total
    logp = torch.gather(z, 2, s["ids"].long()[..., None]).squeeze(-1) - lse
    zero = torch.zeros_like(lse)
    out = [torch.where(act, x, zero) for x in (logp, entropy, lse)]
    if c["top_k"]:
        vals, idx = [], []
        for _ in range(c["top_k"]):
            at = torch.argmax(z, -1, keepdim=True)
            vals.append(torch.gather(z, 2, at))
            idx.append(at)
            z = z.scatter(2, at, float("-inf"))
        vals, idx = torch.cat(vals, -1) - lse[..., None], torch.cat(idx, -1).int()
        out += [torch.where(act[..., None], vals, torch.zeros_like(vals)),
                torch.where(act[..., None], idx, torch.full_like(idx, -1))]
    return out


def _plain_logprobs_bwd(s, c):
    z, act = s["logits"].float(), _active(s)
    lp = z - s["lse"][..., None]
    p = torch.exp(lp)
    up = s["dlogp"][..., None]
    dz = -up * p
    dz.scatter_add_(2, s["ids"].long()[..., None], up)
    if s["dentropy"] is not None:
        dz = dz - s["dentropy"][..., None] * p * (lp + s["entropy"][..., None])
    return (dz * act[..., None]).to(s["logits"].dtype)


def _plain_ortho(U, steps):
    X = U.float()
    flip = X.shape[-2] > X.shape[-1]
    if flip:
        X = X.transpose(-1, -2).contiguous()
    X = X / torch.sqrt((X * X).sum((-2, -1), keepdim=True)).clamp_min(NS_EPS)
    a, b, c = NS_COEFFS
    for _ in range(steps):
        A = torch.matmul(X, X.transpose(-1, -2).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    return X.transpose(-1, -2).contiguous() if flip else X


def _plain_muon(s, c):
    grad, M, W = s["grad"], s["momentum"], s["W"]
    M.mul_(0.95).add_(grad)
    update = _plain_ortho(grad + 0.95 * M, c["steps"])
    W.mul_(1.0 - 0.02 * 0.01).sub_(update * (0.02 * math.sqrt(max(1.0, c["dout"] / c["din"]))))
    return W, M


# ---------------------------------------------------------------------------
def run(state):
    c, op = state["case"], state["op"]
    if not own:
        if op == "lookup":
            return _plain_lookup(state, c)
        if op == "embgrad":
            return _plain_embgrad(state, c)
        if op == "logprobs":
            return _plain_logprobs(state, c)
        if op == "logprobs_bwd":
            return _plain_logprobs_bwd(state, c)
        if op == "ortho":
            return _plain_ortho(state["grad"], c["steps"]).to(state["grad"].dtype)
        return _plain_muon(state, c)
    import sample_gradient_clipping_amd as dp
    if op == "lookup":
        return dp.embedding_lookup(state["ids"], state["table"], mask=state["mask"], scale=c["scale"],
                                   out_dtype=_DT[c["out"]])
    if op == "embgrad":
        return dp.embedding_clip_accumulate(
            state["ids"], state["G"], c["V"], mask=state["mask"], scale=c["scale"], C=state["C"],
            sigma=c["sigma"], seed=state["noise"], offset=7, denom=state["denom"],
            grad_out=state.get("grad"), accumulate=c["accumulate"])
    if op == "logprobs":
        r = dp.token_logprobs(state["logits"], state["ids"], mask=state["mask"], top_k=c["top_k"])
        return [x for x in (r.logp, r.entropy, r.lse, r.top_logp, r.top_ids) if x is not None]
    if op == "logprobs_bwd":
        return dp.token_logprobs_backward(state["logits"], state["ids"], state["lse"], state["dlogp"],
                                          entropy=state["entropy"] if c["entropy"] else None,
                                          dentropy=state["dentropy"], mask=state["mask"])
    if op == "ortho":
        return dp.orthogonalize(state["grad"], steps=c["steps"], coeffs=NS_COEFFS, eps=NS_EPS)
    dp.muon_step(state["grad"], state["momentum"], state["W"], lr=0.02, beta=0.95, nesterov=True,
                 weight_decay=0.01, steps=c["steps"], coeffs=NS_COEFFS, eps=NS_EPS)
    return state["W"], state["momentum"]


# ---------------------------------------------------------------------------
def _distinct(n, V):
    """Expected number of different ids among n tokens of the law in _tokens."""
    v = np.arange(V, dtype=np.float64)
    p = np.log((v + 2) / (v + 1)) / math.log(V + 1.0)
    return float((1 - (1 - p) ** n).sum())


def work(case):
    """Bytes and operations a pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("ortho", "muon"):
        m, n = sorted((case["dout"], case["din"]))
        # both symmetric products need one triangle each
        flops = case["n"] * case["steps"] * (m * m * n + m ** 3 + 2 * m * m * n)
        each = 2 * size[case["dtype"]] if op == "ortho" else 5 * 4
        return {"bytes": each * case["n"] * m * n, "flops": flops}
    N, V = case["B"] * case["T"], case["V"]
    kept = N * (0.53 if case["masked"] else 1.0)  # lengths uniform over (T/16, T)
    b = size[case["dtype"]]
    ids = N * (4 if case["ids"] == "i32" else 8) + (N if case["masked"] else 0)
    if op == "lookup":
        D = case["D"]
        return {"bytes": ids + _distinct(kept, V) * D * b + N * D * size[case["out"]], "flops": kept * D}
    if op == "embgrad":
        D = case["D"]
        table = V * D * 4 * (2 if case["accumulate"] else 1)
        return {"bytes": ids + kept * D * b + table + 4 * case["B"], "flops": 4 * kept * D + V * D}
    if op == "logprobs":
        return {"bytes": ids + kept * V * b + N * (12 + 8 * case["top_k"]), "flops": 6 * kept * V}
    return {"bytes": ids + kept * V * b + N * V * b + N * 12, "flops": 6 * kept * V}


# ---------------------------------------------------------------------------
# The definitions in float64
# ---------------------------------------------------------------------------
def _exact_embgrad(s, c):
    V, D = c["V"], c["D"]
    grad = torch.zeros((V, D), dtype=torch.float64, device="cuda")
    norms = []
    for i in range(c["B"]):
        ids, rows = s["ids"][i].long(), s["G"][i].double()
        if s["mask"] is not None:
            ids, rows = ids[s["mask"][i] != 0], rows[s["mask"][i] != 0]
        words, where = torch.unique(ids, return_inverse=True)
        g = torch.zeros((len(words), D), dtype=torch.float64, device="cuda").index_add_(0, where, rows)
        g *= c["scale"]
        n = float(g.square().sum().sqrt())
        norms.append(n)
        grad[words] += g * (1.0 if n <= s["C"] else s["C"] / n)
    if c["sigma"] > 0:
        grad += c["sigma"] * s["C"] * _philox_normals(s["noise"], 7, V * D).reshape(V, D)
    grad /= s["denom"]
    if c["accumulate"]:
        grad += s["grad"].double()
    return grad, torch.tensor(norms, dtype=torch.float64, device="cuda")


def _exact_logprobs(s, c):
    found = []
    for i in range(c["B"]):
        z = s["logits"][i].double()
        lp = torch.log_softmax(z, -1)
        row = [lp.gather(1, s["ids"][i].long()[:, None])[:, 0], -(lp.exp() * lp).sum(-1),
               torch.logsumexp(z, -1)]
        if c["top_k"]:
            row.append(torch.sort(lp, -1, descending=True).values[:, :c["top_k"]])
        if s["mask"] is not None:
            row = [x * (s["mask"][i] != 0).view(-1, *[1] * (x.dim() - 1)) for x in row]
        found.append(row)
    out = [torch.stack(x) for x in zip(*found)]
    return out + ([None] if c["top_k"] else [])


def _exact_logprobs_bwd(s, c):
    # Only what the definition takes from the call itself: the kept lse and entropy are inputs.
    out = torch.empty((c["B"], c["T"], c["V"]), dtype=torch.float64, device="cuda")
    for i in range(c["B"]):
        lp = s["logits"][i].double() - s["lse"][i].double()[:, None]
        p = lp.exp()
        dz = -s["dlogp"][i].double()[:, None] * p
        t = torch.arange(c["T"], device="cuda")
        dz[t, s["ids"][i].long()] += s["dlogp"][i].double()
        if s["dentropy"] is not None:
            dz -= s["dentropy"][i].double()[:, None] * p * (lp + s["entropy"][i].double()[:, None])
        if s["mask"] is not None:
            dz *= (s["mask"][i] != 0)[:, None]
        out[i] = dz
    return out


def _exact_ortho(U, steps):
    a, b, c = NS_COEFFS
    out = []
    for M in U.reshape(-1, U.shape[-2], U.shape[-1]):
        X = M.double()
        X = X / max(float(X.norm()), NS_EPS)
        for _ in range(steps):
            if X.shape[0] <= X.shape[1]:
                A = X @ X.T
                X = a * X + b * (A @ X) + c * (A @ (A @ X))
            else:
                A = X.T @ X
                X = a * X + b * (X @ A) + c * ((X @ A) @ A)
        out.append(X)
    return torch.stack(out).reshape(U.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        keep = 1.0 if s["mask"] is None else (s["mask"] != 0).double()[..., None]
        return s["table"].double()[s["ids"].long()] * case["scale"] * keep
    if op == "embgrad":
        return _exact_embgrad(s, case)
    if op == "logprobs":
        return _exact_logprobs(s, case)
    if op == "logprobs_bwd":
        return _exact_logprobs_bwd(s, case)
    if op == "ortho":
        return _exact_ortho(s["grad"], case["steps"])
    g, M, W = s["grad"].double(), s["momentum"].double(), s["W"].double()
    M = 0.95 * M + g
    size = 0.02 * math.sqrt(max(1.0, case["dout"] / case["din"]))
    return (1.0 - 0.02 * 0.01) * W - size * _exact_ortho(g + 0.95 * M, case["steps"]), M
