"""One block of a transformer trained with DP-SGD on packed documents, one clip
factor per row over all its weights, norms included, then asked for tokens one
at a time over a cache:

    X = embedding rows of the tokens               embedding_lookup
    q, k, v = X Wqkv^T                             plain matrix product
    q, k: norms per head, rotated by position      qk_norm_rotary
    A = attention within each document             attention
    R = X + dropout(A Wo^T)                        dropout
    log p(next token), logits = R W^T              token_logprobs

and backwards with token_logprobs_backward, dropout (the same mask, drawn
again), attention_backward and qk_norm_rotary_backward, which leave dq, dk and dv
as parts of one array: the G of Wqkv's private gradient.  The norms' weights get
their per-sample gradients as a linear of one input.

The data are synthetic: a document repeats a random phrase; a row packs two.

    python examples/private_transformer.py [--steps 60] [--sigma 0.2]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import sample_gradient_clipping_amd as dp  # noqa: E402

LINEARS = ("wqkv", "wo", "w")
NORMS = ("q_norm", "k_norm")


def make_model(V, width, Hq, Hkv, D, seed=0, device="cuda"):
    """float32 master weights, the rotation's frequencies and its amplitude."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s, scale: (torch.randn(s, generator=g) * scale).to(device)  # noqa: E731
    freqs, amplitude = dp.rotary_frequencies(D // 2 * 2, device=device)
    return {"heads": (Hq, Hkv, D), "freqs": freqs, "amplitude": amplitude,
            "table": draw(V, width, scale=1.0),
            "wqkv": draw((Hq + 2 * Hkv) * D, width, scale=width ** -0.5),
            "wo": draw(width, Hq * D, scale=(Hq * D) ** -0.5), "w": draw(V, width, scale=width ** -0.5),
            "q_norm": torch.ones(D, device=device), "k_norm": torch.ones(D, device=device)}


def make_batch(B, T, V, generator, phrase=5):
    """ids, next tokens, documents, positions [B, T], and the weight of each token's loss: the mean
    over a row's tokens but each document's last."""
    ids = torch.empty((B, T), dtype=torch.int64)
    cuts = torch.randint(2, T - 1, (B,), generator=generator)
    for b in range(B):
        c = int(cuts[b])
        for at, n in ((0, c), (c, T - c)):
            words = torch.randint(0, V, (phrase,), generator=generator)
            ids[b, at:at + n] = words.repeat(n // phrase + 1)[:n]
    t = torch.arange(T)[None, :]
    documents = (t >= cuts[:, None]).to(torch.int32)
    positions = t - documents * cuts[:, None]
    counts = ((t + 1 < T) & (t + 1 != cuts[:, None])).float()
    weight = counts / counts.sum(dim=1, keepdim=True)
    targets = ids.roll(-1, 1)
    return tuple(x.contiguous().cuda() for x in (ids, targets, documents, positions, weight))


def rows_times(X, W):
    """X [B, T, k] times W [k, n], as one matrix product."""
    return (X.reshape(-1, X.shape[2]) @ W).reshape(X.shape[0], X.shape[1], W.shape[1])


def split(qkv, heads):
    """Queries [B, T, Hq, D], keys and values [B, T, Hkv, D] as parts of a projection's output."""
    Hq, Hkv, D = heads
    parts = qkv.view(qkv.shape[0], qkv.shape[1], Hq + 2 * Hkv, D)
    return parts[:, :, :Hq], parts[:, :, Hq:Hq + Hkv], parts[:, :, Hq + Hkv:]


def project(model, ids, positions, dtype):
    """Embedded tokens, the projection as it is and its queries and keys after their norms."""
    X = dp.embedding_lookup(ids, model["table"], out_dtype=dtype)
    qkv = rows_times(X, model["wqkv"].to(dtype).t())
    q, k, _ = split(qkv, model["heads"])
    return X, qkv, dp.qk_norm_rotary(q, k, model["q_norm"], model["k_norm"], model["freqs"], positions,
                                     amplitude=model["amplitude"])


def private_gradients(model, batch, C, sigma, seed, p=0.1, dtype=torch.bfloat16):
    """The clipped and noised mean gradient of each weight, the rows' norms, and the log
    probabilities of the next tokens."""
    ids, targets, documents, positions, weight = batch
    B, T = ids.shape
    heads = model["heads"]
    X, qkv, (q, k) = project(model, ids, positions, dtype)
    v = split(qkv, heads)[2]
    att = dp.attention(q, k, v, segments=documents)
    A = att.out.reshape(B, T, -1)
    R = dp.dropout(rows_times(A, model["wo"].to(dtype).t()), p, seed, residual=X)
    logits = rows_times(R, model["w"].to(dtype).t())
    out = dp.token_logprobs(logits, targets)

    dlogits = dp.token_logprobs_backward(logits, targets, out.lse, -weight, out=logits)
    dR = rows_times(dlogits, model["w"].to(dtype))
    dY = dp.dropout(dR, p, seed)
    dA = rows_times(dY, model["wo"].to(dtype)).view(att.out.shape)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = split(dqkv, heads)
    dp.attention_backward(dA, q, k, v, att.out, att.lse, segments=documents, dq=dq, dk=dk, dv=dv)
    before = split(qkv, heads)
    norm = dp.qk_norm_rotary_backward(dq, dk, before[0], before[1], model["q_norm"], model["k_norm"],
                                      model["freqs"], positions, amplitude=model["amplitude"], dq=dq, dk=dk)
    dX = rows_times(dqkv, model["wqkv"].to(dtype)).add_(dR)

    V, one = model["table"].shape[0], torch.ones((B, 1, 1), dtype=torch.float32, device=ids.device)
    pairs = {"wqkv": (X, dqkv), "wo": (A, dY), "w": (R, dlogits), "q_norm": (one, norm.dq_weight),
             "k_norm": (one, norm.dk_weight)}
    squared = dp.embedding_sqnorms(ids, dX, V)
    for x, g in pairs.values():
        dp.per_sample_sqnorms(x, g, out=squared, accumulate=True)
    norms = torch.empty(B, dtype=torch.float32, device=ids.device)
    c, norms = dp.clip_factors(squared, C, norms_out=norms)
    # each weight draws its own stretch of the step's noise
    shapes = [(g.shape[2], x.shape[2]) for x, g in pairs.values()]
    at = dp.consecutive_offsets([tuple(model["table"].shape), *shapes])
    noise = dict(noise_std=sigma * C, seed=seed)
    grads = {"table": dp.embedding_scaled_accumulate(ids, dX, c, V, offset=at[0], **noise)}
    for offset, (name, (x, g)) in zip(at[1:], pairs.items()):
        grads[name] = dp.scaled_accumulate(x, g, c, offset=offset, **noise).view(model[name].shape)
    return grads, norms, out


def next_logits(model, ids, cache, length, dtype=torch.bfloat16):
    """Logits of the last of the new tokens ids [B, n], the first of them at position ``length``:
    their keys and values join the cache ([B, room, Hkv, D] each), their queries see all of it."""
    B, n = ids.shape
    positions = torch.arange(length, length + n, device=ids.device).expand(B, n).contiguous()
    X, qkv, (q, k) = project(model, ids, positions, dtype)
    keys, values = cache
    keys[:, length:length + n] = k
    values[:, length:length + n] = split(qkv, model["heads"])[2]
    att = dp.attention(q, keys[:, :length + n], values[:, :length + n])
    R = X + rows_times(att.out.reshape(B, n, -1), model["wo"].to(dtype).t())
    return rows_times(R[:, -1:], model["w"].to(dtype).t())


def generate(model, ids, count, dtype=torch.bfloat16):
    """The ``count`` most likely tokens after ids [B, n], one at a time."""
    _, Hkv, D = model["heads"]
    room = (ids.shape[0], ids.shape[1] + count, Hkv, D)
    cache = [torch.empty(room, dtype=dtype, device=ids.device) for _ in range(2)]
    out, new, length = [], ids, 0
    for _ in range(count):
        logits = next_logits(model, new, cache, length, dtype)
        length += new.shape[1]
        new = dp.token_logprobs(logits, top_k=1).top_ids[:, :, 0].to(torch.int64)
        out.append(new)
    return torch.cat(out, dim=1)


def train(steps=60, B=256, T=48, V=128, width=128, Hq=4, Hkv=2, D=32, C=1.0, sigma=0.2, lr=0.02,
          table_lr=4.0, norm_lr=0.1, log=print):
    """Trains for ``steps`` steps; the mean loss of each."""
    model = make_model(V, width, Hq, Hkv, D)
    momentum = {k: torch.zeros_like(model[k]) for k in LINEARS}
    generator = torch.Generator().manual_seed(1)
    losses = []
    for step in range(steps):
        batch = make_batch(B, T, V, generator)
        grads, norms, out = private_gradients(model, batch, C, sigma, seed=step)
        model["table"].sub_(grads["table"], alpha=table_lr)
        for k in NORMS:
            model[k].sub_(grads[k], alpha=norm_lr)
        for k in LINEARS:
            dp.muon_step(grads[k], momentum[k], model[k], lr)
        losses.append(float(-(out.logp * batch[4]).sum() / B))
        if step % 10 == 0 or step + 1 == steps:
            log(f"step {step:4d}  loss {losses[-1]:.3f}  perplexity {math.exp(losses[-1]):8.1f}  "
                f"clipped {float((norms > C).float().mean()):.2f} of the rows")
    ids = make_batch(4, 16, V, generator)[0]
    for row, tokens in zip(ids[:, 8:].tolist(), generate(model, ids, 8).tolist()):
        log(f"after {row}: {tokens}")
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--sigma", type=float, default=0.2)
    args = parser.parse_args()
    train(steps=args.steps, sigma=args.sigma)
