"""fp64 reference of the operators between a language model's linears: attention, the norms and
rotation of queries and keys, dropout, and their gradients, straight from the definitions.

Arrays are [B, T, heads, D].  Beside the values the attention functions give what bounds the
rounding of a float32 computation of them.  Nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

from .philox import MASK32, philox4x32_10, seed_key

U = 2.0 ** -24                                    # half a step of float32
HALF = {"f32": U, "bf16": 2.0 ** -8}              # of the type, relative


def allowed(b, Tq, Tk, mask, segments, causal):
    """[Tq, Tk] truth values of sample b: the query attends to the key."""
    p, j = np.arange(Tk - Tq, Tk)[:, None], np.arange(Tk)[None, :]
    ok = np.ones((Tq, Tk), bool)
    if causal:
        ok &= j <= p
    if segments is not None:
        ok &= segments[b][p] == segments[b][j]
    if mask is not None:
        ok &= (mask[b][p] != 0) & (mask[b][j] != 0)
    return ok


def oracle_attention(q, k, v, mask, segments, causal, scale, dtype, dout=None):
    """out, lse and, with dout, dq, dk, dv; each with a bar of the same shape.

    The bars follow the computation: scores are sums of D products, off by (D + 4) u of the sum of
    their magnitudes A; a weight e^(s - m) by the errors of s and m and 8 u; sums over n terms by
    (n + 16) u of the sum of magnitudes; weights and dS are rounded to the inputs' type (half a
    step) before their products, results once more; delta comes from the rounded output."""
    B, Tq, Hq, D = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    step, narrow = HALF[dtype], (HALF[dtype] if dtype == "bf16" else 0.0)
    out, t_out = np.zeros(q.shape), np.zeros(q.shape)
    lse, t_lse = np.zeros((B, Hq, Tq)), np.zeros((B, Hq, Tq))
    back = dout is not None
    dq, t_dq = np.zeros(q.shape), np.zeros(q.shape)
    dk, dv, t_dk, t_dv = (np.zeros(k.shape) for _ in range(4))
    m_dk, m_dv = np.zeros(k.shape), np.zeros(k.shape)
    for b in range(B):
        ok = allowed(b, Tq, Tk, mask, segments, causal)
        live = ok.any(1)
        if not live.any():
            continue
        for h in range(Hq):
            g = h * Hkv // Hq
            # places that are masked out may hold anything
            Q = np.where(live[:, None], q[b, :, h], 0.0)
            seen = ok.any(0)[:, None]
            K, V = np.where(seen, k[b, :, g], 0.0), np.where(seen, v[b, :, g], 0.0)
            s = np.where(ok, scale * (Q @ K.T), -np.inf)
            A = np.where(ok, abs(scale) * (np.abs(Q) @ np.abs(K).T), 0.0)
            m = np.where(live, s.max(1), 0.0)
            w = np.exp(s - m[:, None])
            total = w.sum(1)
            L = np.where(live, m + np.log(np.where(live, total, 1.0)), 0.0)
            P = w / np.where(live, total, 1.0)[:, None]
            O = P @ V
            e_s = (D + 6) * U * A.max(1) + 4 * U * np.abs(m)
            e_w = 2 * e_s + 8 * U
            mag = P @ np.abs(V)
            e_o = mag * (2 * e_w + (2 * Tk + 32) * U + narrow)[:, None]
            out[b, :, h], t_out[b, :, h] = O, e_o + step * (np.abs(O) + e_o)
            lse[b, h] = L
            t_lse[b, h] = np.where(live, 2 * e_w + (Tk + 16) * U + 6 * U * (np.abs(L) + np.abs(m) + 1), 0.0)
            if not back:
                continue
            G = np.where(live[:, None], dout[b, :, h], 0.0)
            e_p = (e_s + t_lse[b, h] + 8 * U * (1 + np.abs(L)))[:, None]
            dP = G @ V.T
            delta = (G * O).sum(1)[:, None]
            e_dP = (D + 4) * U * (np.abs(G) @ np.abs(V).T)
            e_delta = (np.abs(G) * (t_out[b, :, h] + (D + 4) * U * np.abs(O))).sum(1)[:, None]
            dS = P * (dP - delta)
            dS[ok.sum(1) == 1] = 0.0
            e_dS = P * ((np.abs(dP) + np.abs(delta)) * e_p + e_dP + e_delta)
            e_dS += narrow * (np.abs(dS) + e_dS)
            N = Tq * (Hq // Hkv)
            dq[b, :, h] = scale * dS @ K
            e = scale * (e_dS @ np.abs(K) + (Tk + 16) * U * (np.abs(dS) @ np.abs(K)))
            t_dq[b, :, h] = e + step * (np.abs(dq[b, :, h]) + e)
            dk[b, :, g] += scale * dS.T @ Q
            m_dk[b, :, g] += scale * (e_dS.T @ np.abs(Q) + (N + 16) * U * (np.abs(dS).T @ np.abs(Q)))
            dv[b, :, g] += P.T @ G
            m_dv[b, :, g] += (P * (e_p + narrow)).T @ np.abs(G) * 1.01 + (N + 16) * U * (P.T @ np.abs(G))
    if not back:
        return (out, t_out), (lse, t_lse)
    return ((out, t_out), (lse, t_lse), (dq, t_dq), (dk, m_dk + step * (np.abs(dk) + m_dk)),
            (dv, m_dv + step * (np.abs(dv) + m_dv)))


def _rotate(x, cos, sin, pairs, interleaved):
    y = x.copy()
    a, b = (x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]) if interleaved else \
        (x[..., :pairs], x[..., pairs:2 * pairs])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2] = lo, hi
    else:
        y[..., :pairs], y[..., pairs:2 * pairs] = lo, hi
    return y


def oracle_rotary(x, w, eps, freqs, positions, amplitude, interleaved, mask, dy=None):
    """The normalised (w not None) and rotated heads, or with dy the gradients to x and to w per
    sample ([B, D], None without w); each with its bar.

    Bars: r is good to (D / 2 + 8) u, cosines and sines to 8 u absolute, each product and sum one u
    more; sums of n terms (n + 16) u of their magnitudes; no rounding of results."""
    B, T, H, D = x.shape
    pairs = len(freqs)
    t = np.broadcast_to(np.arange(T), (B, T)) if positions is None else positions
    angle = t[..., None, None].astype(np.float64) * np.asarray(freqs)
    cos, sin = amplitude * np.cos(angle), amplitude * np.sin(angle)
    live = np.ones((B, T), bool) if mask is None else mask != 0
    keep = live[..., None, None]
    x = np.where(keep, x, 0.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    size = max(1.0, abs(amplitude))
    c_n, c_t = (D / 2 + 12) * U, 16 * U * size
    one = np.ones_like(cos)
    # magnitudes of an entry and of its pair's two
    around = lambda z: z + np.maximum(_rotate(z, one, one, pairs, interleaved),  # noqa: E731
                                      _rotate(z, one, -one, pairs, interleaved))
    if dy is None:
        y = x if w is None else n * w
        bar = around(np.abs(y)) * (size * c_n + c_t)
        return np.where(keep, _rotate(y, cos, sin, pairs, interleaved), 0.0), np.where(keep, bar, 0.0)
    dy = np.where(keep, dy, 0.0)
    d = np.where(keep, _rotate(dy, cos, -sin, pairs, interleaved), 0.0)
    e_d = np.where(keep, around(np.abs(dy)) * c_t, 0.0)
    if w is None:
        return d, e_d + U * np.abs(d), None, None
    dw, e_dw = d * w, e_d * np.abs(w) + 2 * U * np.abs(d * w)
    mean = (dw * n).mean(-1, keepdims=True)
    e_mean = ((np.abs(dw) * (c_n + (D + 16) * U) + e_dw) * np.abs(n)).mean(-1, keepdims=True)
    dx = r * (dw - n * mean)
    bar = r * (e_dw + np.abs(n) * (e_mean + 4 * U * np.abs(mean) + c_n * np.abs(mean))
               + (c_n + 4 * U) * (np.abs(dw) + np.abs(n * mean)))
    gw = (d * n).sum((1, 2))
    t_gw = ((np.abs(d) * (c_n + (T * H + 16) * U) + e_d) * np.abs(n)).sum((1, 2))
    return np.where(keep, dx, 0.0), np.where(keep, bar, 0.0), gw, t_gw


def dropout_bits(seed, offset, n):
    """The 16 random bits of entries 0 .. n - 1, one block at a time from the definition."""
    bits = []
    for j in range((n + 7) // 8):
        block = (offset + j) & ((1 << 64) - 1)
        for word in philox4x32_10((block & MASK32, block >> 32, 1, 0), seed_key(seed)):
            bits += [word & 0xFFFF, word >> 16]
    return np.array(bits[:n], np.int64)


def oracle_dropout(x, p, seed, offset, residual, mask):
    """(y, kept) in float64."""
    limit = round(p * 65536)
    kept = (dropout_bits(seed, offset, x.size) >= limit).reshape(x.shape)
    live = np.ones(x.shape[:2], bool) if mask is None else mask != 0
    with np.errstate(all="ignore"):
        y = np.where(kept, x * (65536.0 / (65536 - limit)), 0.0)
    if residual is not None:
        y = y + residual
    return np.where(live[..., None], y, 0.0), kept
