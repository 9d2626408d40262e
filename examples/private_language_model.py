"""A small language model trained with DP-SGD, one clip factor per sample over
all its layers (group clipping):

    X = embedding rows of the tokens          embedding_lookup
    H = relu(X W1^T),  logits = H W2^T        plain matrix products
    log p(next token)                         token_logprobs
    d loss / d logits                         token_logprobs_backward
    ||g_i||^2 over the three layers           embedding_sqnorms, per_sample_sqnorms
    c_i = min(1, C / ||g_i||)                 clip_factors
    clipped, noised gradients                 embedding_scaled_accumulate, scaled_accumulate
    update of the two weights, of the table   muon_step, plain descent

The data are synthetic: token t is followed by (7 t + 3) mod V nine times of
ten and by a random one otherwise, sentences have random lengths.

    python examples/private_language_model.py [--steps 60] [--sigma 0.4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import sample_gradient_clipping_amd as dp  # noqa: E402


def make_model(V, D, H, seed=0, device="cuda"):
    """float32 master weights: the table [V, D], W1 [H, D] and W2 [V, H]."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s, scale: (torch.randn(s, generator=g) * scale).to(device)  # noqa: E731
    return {"table": draw(V, D, scale=1.0), "w1": draw(H, D, scale=D ** -0.5),
            "w2": draw(V, H, scale=H ** -0.5)}


def make_batch(B, T, V, generator):
    """ids, next tokens [B, T] and the mask of the sentences' tokens."""
    ids = torch.empty((B, T + 1), dtype=torch.int64)
    ids[:, 0] = torch.randint(0, V, (B,), generator=generator)
    for t in range(T):
        jump = torch.rand(B, generator=generator) < 0.1
        ids[:, t + 1] = torch.where(jump, torch.randint(0, V, (B,), generator=generator),
                                    (7 * ids[:, t] + 3) % V)
    lengths = torch.randint(T // 2, T + 1, (B,), generator=generator)
    mask = (torch.arange(T)[None, :] < lengths[:, None]).to(torch.uint8)
    return ids[:, :T].contiguous().cuda(), ids[:, 1:].contiguous().cuda(), mask.cuda()


def rows_times(X, W):
    """X [B, T, k] times W [k, n], as one matrix product."""
    return (X.reshape(-1, X.shape[2]) @ W).reshape(X.shape[0], X.shape[1], W.shape[1])


def forward(model, ids, mask, dtype):
    """The embedded tokens, the hidden layer and the logits, in ``dtype``."""
    X = dp.embedding_lookup(ids, model["table"], mask=mask, out_dtype=dtype)
    H = torch.relu(rows_times(X, model["w1"].to(dtype).t()))
    return X, H, rows_times(H, model["w2"].to(dtype).t())


def private_gradients(model, ids, targets, mask, C, sigma, seed, dtype=torch.bfloat16):
    """The clipped and noised mean gradient of each layer, the samples' norms, and the log
    probabilities of the next tokens.  A sample's loss is its tokens' mean."""
    X, H, logits = forward(model, ids, mask, dtype)
    out = dp.token_logprobs(logits, targets, mask=mask)
    weight = -1.0 / mask.sum(dim=1, keepdim=True).clamp(min=1).float()
    dlogits = dp.token_logprobs_backward(logits, targets, out.lse, weight.expand(ids.shape).contiguous(),
                                         mask=mask, out=logits)
    dH = rows_times(dlogits, model["w2"].to(dtype)) * (H > 0)
    dX = rows_times(dH, model["w1"].to(dtype))
    V = model["table"].shape[0]
    squared = dp.embedding_sqnorms(ids, dX, V, mask=mask)
    dp.per_sample_sqnorms(X, dH, mask=mask, out=squared, accumulate=True)
    dp.per_sample_sqnorms(H, dlogits, mask=mask, out=squared, accumulate=True)
    norms = torch.empty(ids.shape[0], dtype=torch.float32, device=ids.device)
    c, norms = dp.clip_factors(squared, C, norms_out=norms)
    # each layer draws its own stretch of the step's noise
    at = dp.consecutive_offsets([tuple(model[k].shape) for k in ("table", "w1", "w2")])
    noise = dict(noise_std=sigma * C, seed=seed)
    grads = {"table": dp.embedding_scaled_accumulate(ids, dX, c, V, mask=mask, offset=at[0], **noise),
             "w1": dp.scaled_accumulate(X, dH, c, mask=mask, offset=at[1], **noise),
             "w2": dp.scaled_accumulate(H, dlogits, c, mask=mask, offset=at[2], **noise)}
    return grads, norms, out


def train(steps=60, B=256, T=32, V=512, D=128, H=256, C=1.0, sigma=0.4, lr=0.02, table_lr=4.0,
          log=print):
    """Trains for ``steps`` steps; the mean loss of each."""
    model = make_model(V, D, H)
    momentum = {k: torch.zeros_like(model[k]) for k in ("w1", "w2")}
    generator = torch.Generator().manual_seed(1)
    losses = []
    for step in range(steps):
        ids, targets, mask = make_batch(B, T, V, generator)
        grads, norms, out = private_gradients(model, ids, targets, mask, C, sigma, seed=step)
        model["table"].sub_(grads["table"], alpha=table_lr)
        for k in ("w1", "w2"):
            dp.muon_step(grads[k], momentum[k], model[k], lr)
        losses.append(float(-out.logp.sum() / mask.sum()))
        if step % 10 == 0 or step + 1 == steps:
            log(f"step {step:4d}  loss {losses[-1]:.3f}  perplexity {math.exp(losses[-1]):8.1f}  "
                f"entropy {float(out.entropy.sum() / mask.sum()):.3f}  "
                f"clipped {float((norms > C).float().mean()):.2f} of the samples")
    ids = torch.arange(8, device="cuda").reshape(8, 1)
    _, _, logits = forward(model, ids, None, torch.bfloat16)
    best = dp.token_logprobs(logits, top_k=3)
    for i in range(8):
        log(f"after {i}: " + ", ".join(f"{int(k)} ({math.exp(float(p)):.2f})" for k, p in
                                        zip(best.top_ids[i, 0], best.top_logp[i, 0])))
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--sigma", type=float, default=0.4)
    args = parser.parse_args()
    train(steps=args.steps, sigma=args.sigma)
