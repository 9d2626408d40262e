"""Gradients of bf16 attention over few keys, where delta_i = sum_j P_ij dO_i . v_j is summed from the
weights: from the rounded output it would be off by half a step of |dO| |O|, which is much more than dS
where the values are nearly alike.  Against float64, with a bar that has no room for that half step."""
import numpy as np
import pytest

from oracle import attention as oracle
from oracle.dp_linear import widen
from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U, STEP = oracle.U, oracle.HALF["bf16"]


def _reference(q, k, v, dout, ok, rounded=None):
    """(dq, dk) of one sample [T, H, D] and their bars; with ``rounded`` (the output as it is stored)
    delta comes from that.

    Roundings, u = 2^-24: scores D products, weights e^(s - lse) as in oracle_attention; dO . v - delta
    starts from -delta: (D + 6) u of |dO| |v| + |delta|; delta = d0 + sum_j P_ij (dO . v_j - d0), d0 the
    rounded output's, off by n: its sum's error (T + 16) u and the weights' errors count for
    |dO . v_j - delta| + n, and the result is rounded once (u |delta|); dS and the results to bf16."""
    T, H, D = q.shape
    scale = D ** -0.5
    dq, dk, t_dq, m_dk = (np.zeros(q.shape) for _ in range(4))
    for h in range(H):
        Q, K, V, G = q[:, h], k[:, h], v[:, h], dout[:, h]
        s = np.where(ok, scale * (Q @ K.T), -np.inf)
        A = np.where(ok, scale * (np.abs(Q) @ np.abs(K).T), 0.0)
        m = s.max(1)
        w = np.exp(s - m[:, None])
        L = m + np.log(w.sum(1))
        P = np.exp(s - L[:, None])
        e_s = (D + 6) * U * A.max(1) + 4 * U * np.abs(m)
        e_w = 2 * e_s + 8 * U
        t_lse = 2 * e_w + (T + 16) * U + 6 * U * (np.abs(L) + np.abs(m) + 1)
        e_p = (e_s + t_lse + 8 * U * (1 + np.abs(L)))[:, None]
        O = P @ V
        dP, delta = G @ V.T, (G * O).sum(1)[:, None]
        t_out = (P @ np.abs(V)) * (2 * e_w + (2 * T + 32) * U + STEP)[:, None] + STEP * np.abs(O) * 1.01
        n = (np.abs(G) * (t_out + (D + 4) * U * np.abs(O))).sum(1)[:, None]
        far = np.abs(dP - delta)
        e_dP = (D + 6) * U * (np.abs(G) @ np.abs(V).T + np.abs(delta) + n)
        e_delta = (P * ((far + n) * (e_p + (T + 16) * U) + e_dP)).sum(1)[:, None] + 2 * U * (np.abs(delta) + n)
        if rounded is not None:
            delta = (G * rounded[:, h]).sum(1)[:, None]
        dS = P * (dP - delta)
        dS[ok.sum(1) == 1] = 0.0
        e_dS = P * (far * e_p + e_dP + e_delta)
        e_dS += STEP * (np.abs(dS) + e_dS)
        dq[:, h], dk[:, h] = scale * dS @ K, scale * dS.T @ Q
        e = scale * (e_dS @ np.abs(K) + (T + 16) * U * (np.abs(dS) @ np.abs(K)))
        t_dq[:, h] = e + STEP * (np.abs(dq[:, h]) + e)
        m_dk[:, h] = scale * (e_dS.T @ np.abs(Q) + (T + 16) * U * (np.abs(dS).T @ np.abs(Q)))
    return dq, t_dq, dk, m_dk + STEP * (np.abs(dk) + m_dk)


# The first's waves share 32 queries (up to four tiles of 32 keys), the others have 32 each (a tile of 64).
@pytest.mark.parametrize("B,T,H", [(2, 30, 2), (2, 100, 2), (1, 128, 2), (80, 20, 2), (80, 64, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 45, 128])
def test_delta_is_summed_from_the_weights(D, causal, B, T, H):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(T + D)
    q, k, dout = (rng.standard_normal((B, T, H, D)) for _ in range(3))
    v = 1.37 + rng.standard_normal((B, T, H, D)) / 64          # nearly alike
    bits = [f32_to_bf16_bits(x.astype(np.float32)) for x in (q, k, v, dout)]
    tq, tk, tv, td = (to_dev(x, "bf16", torch) for x in bits)
    r = dp.attention(tq, tk, tv, causal=causal)
    grads = dp.attention_backward(td, tq, tk, tv, r.out, r.lse, causal=causal)
    torch.cuda.synchronize()
    got_q, got_k = (x.double().cpu().numpy() for x in grads[:2])
    stored = r.out.double().cpu().numpy()
    wide = [widen(x, "bf16") for x in bits]
    ok = np.tri(T, dtype=bool) if causal else np.ones((T, T), bool)
    for b in range(min(B, 3)):
        one = [x[b] for x in wide]
        dq, t_dq, dk, t_dk = _reference(*one, ok)
        for name, got, want, bar in (("dq", got_q[b], dq, t_dq), ("dk", got_k[b], dk, t_dk)):
            err = np.abs(got - want)
            fine = bool(np.isfinite(err).all() and (err <= bar).all())
            assert fine, (b, name, float((err / bar).max()))
        # the rounded output's delta, in the reference, does not stay within the bars
        lost = _reference(*one, ok, rounded=stored[b])
        assert (np.abs(lost[0] - dq) > 2 * t_dq).any() and (np.abs(lost[2] - dk) > 2 * t_dk).any()
