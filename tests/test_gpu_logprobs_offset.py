"""Log probabilities do not change when a row's logits move together.

Logits are multiples of 1/64 up to 16 in size, and the offsets are powers of two that leave every
sum exact, so both rows have the same differences to their maximum.  Bars, u = 2^-24: those of
tests/test_gpu_logprobs.py for log S, without any term in the logits' size.
"""
import numpy as np
import pytest

from oracle.language_model import oracle_logprobs
from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("offset", [0.0, 2.0 ** 10, 2.0 ** 15, -2.0 ** 15, -2.0 ** 17])
@pytest.mark.parametrize("shape", [(2, 3, 40), (1, 5, 5000), (1, 2, 300001), (40, 70, 2100)])
def test_a_common_offset_changes_nothing(shape, offset):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V = shape
    rng = np.random.default_rng(V)
    z = (rng.integers(-1024, 1025, shape) / 64).astype(np.float32)
    y = rng.integers(0, V, (B, T))
    moved = z + np.float32(offset)
    assert np.array_equal(moved.astype(np.float64), z.astype(np.float64) + offset)
    r = dp.token_logprobs(torch.from_numpy(moved).cuda(), torch.from_numpy(y).cuda(), top_k=4)
    base = dp.token_logprobs(torch.from_numpy(z).cuda(), torch.from_numpy(y).cuda(), top_k=4)
    for got, same in ((r.logp, base.logp), (r.entropy, base.entropy), (r.top_logp, base.top_logp),
                      (r.top_ids, base.top_ids)):
        assert torch.equal(got, same)
    logp, _, lse, top, ids = oracle_logprobs(z.astype(np.float64), y, None, 4)
    d = z.max(-1, keepdims=True).astype(np.float64) - z
    p = np.exp(-d)
    S = p.sum(-1)
    dbar = (p * d).sum(-1) / S
    t = U * (V / 64 + 64 + 4 + dbar + 2 * np.log(S) + 2)     # of log S
    err = np.abs(r.logp.cpu().numpy() - logp)
    assert (err <= t + 2 * U * np.abs(logp)).all(), float(err.max())
    err = np.abs(r.top_logp.cpu().numpy() - top)
    assert (err <= t[..., None] + 2 * U * np.abs(top)).all(), float(err.max())
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    want = lse + offset
    assert (np.abs(r.lse.cpu().numpy() - want) <= t + 2 * U * np.abs(want)).all()


def test_equal_lowest_values():
    """A row of the type's lowest value: every logit has probability 1 / V."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for dtype in (torch.float32, torch.bfloat16):
        for V in (1, 37, 4096, 50257):
            z = torch.full((1, 2, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
            y = torch.tensor([[0, V - 1]], device="cuda")
            r = dp.token_logprobs(z, y, top_k=1)
            bar = U * (V / 64 + 64 + 4 + 2 * np.log(V) + 2) + 2 * U * np.log(V)
            for x in (r.logp, r.top_logp[..., 0], -r.entropy):
                assert float((x.double() + np.log(V)).abs().max()) <= bar
