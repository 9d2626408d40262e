"""fp64 reference of the operators at a language model's two ends.

Embedding: every per-sample gradient is formed explicitly, one dense [V, D]
array per sample, then clipped, summed and noised, straight from the
definition.  Token log probabilities: a softmax in float64, its gradient, and
the alternatives by a full sort.  Nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

from .philox import gaussian


def active_positions(ids, mask, V):
    """[B, T] truth values: the mask byte is not 0 and the id is in [0, V)."""
    act = (ids >= 0) & (ids < V)
    return act if mask is None else act & (np.asarray(mask) != 0)


def oracle_embedding(ids, G, mask, V, scale, C, sigma, seed, offset, denom):
    """(grad [V, D], norms [B], abs_sum [V, D]): the last is (sum_i c_i scale sum_t |G_it|) / denom,
    which scales the rounding of the sums."""
    B, T, D = G.shape
    act = active_positions(ids, mask, V)
    total, mag = np.zeros((V, D)), np.zeros((V, D))
    norms = np.zeros(B)
    for i in range(B):
        g, m = np.zeros((V, D)), np.zeros((V, D))
        for t in range(T):
            if act[i, t]:
                g[ids[i, t]] += scale * G[i, t]
                m[ids[i, t]] += abs(scale) * np.abs(G[i, t])
        norms[i] = np.sqrt((g * g).sum())
        c = 1.0 if norms[i] <= C else C / norms[i]
        total += c * g
        mag += c * m
    if sigma > 0:
        total = total + sigma * C * gaussian(seed, offset, V * D).reshape(V, D)
    return total / denom, norms, mag / denom


def oracle_logprobs(z, targets, mask, top_k):
    """(logp, entropy, lse, top_logp, top_ids) of logits z [B, T, V] in float64."""
    B, T, V = z.shape
    m = z.max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        e = np.exp(z - m)
        S = e.sum(-1)
        lse = m[..., 0] + np.log(S)
        p = e / S[..., None]
        entropy = -np.where(p > 0, p * np.log(np.where(p > 0, p, 1.0)), 0.0).sum(-1)
    inside = (targets >= 0) & (targets < V)
    at = np.where(inside, targets, 0)
    logp = np.where(inside, np.take_along_axis(z, at[..., None], -1)[..., 0] - lse, 0.0)
    order = np.argsort(-z, axis=-1, kind="stable")[..., :top_k]
    top = np.take_along_axis(z, order, -1) - lse[..., None]
    ids = order.astype(np.int64)
    if mask is not None:
        keep = np.asarray(mask) != 0
        logp, entropy, lse = (np.where(keep, x, 0.0) for x in (logp, entropy, lse))
        top = np.where(keep[..., None], top, 0.0)
        ids = np.where(keep[..., None], ids, -1)
    return logp, entropy, lse, top, ids


def oracle_logprobs_grad(z, targets, mask, lse, entropy, dlogp, dentropy):
    """dz [B, T, V] in float64 from the given lse and entropy."""
    B, T, V = z.shape
    lp = z - lse[..., None]
    p = np.exp(lp)
    dz = np.zeros_like(z)
    if dlogp is not None:
        inside = (targets >= 0) & (targets < V)
        up = np.where(inside, dlogp, 0.0)
        dz -= up[..., None] * p
        b, t = np.nonzero(inside)
        dz[b, t, targets[b, t]] += up[b, t]
    if dentropy is not None:
        q = np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + entropy[..., None]), 0.0)
        dz -= dentropy[..., None] * q
    if mask is not None:
        dz *= (np.asarray(mask) != 0)[..., None]
    return dz
