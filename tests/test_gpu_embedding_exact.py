"""The embedding's norms and sums where float32 is exact.

Integers (tests/embedding_integers.py): no sum rounds, so gradients are compared bit for bit, and
a norm has float64's square root and one rounding to float32: 2 u, u = 2^-24.
"""
import numpy as np
import pytest

from tests.embedding_integers import CASES, exact_sums, make_case
from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev(torch, ids, G, mask, dtype):
    return (torch.from_numpy(ids).cuda(),
            to_dev(f32_to_bf16_bits(G) if dtype == "bf16" else G, dtype, torch),
            None if mask is None else torch.from_numpy(mask).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_integers_are_exact(case, dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V, D, _ = case
    ids, G, mask = make_case(*case)
    sums = exact_sums(ids, G, mask, V)
    norms = np.sqrt((sums ** 2).sum((1, 2)))
    i, g, m = _dev(torch, ids, G, mask, dtype)
    # nothing clipped, a power of two as the divisor
    out, n = dp.embedding_clip_accumulate(i, g, V, mask=m, scale=0.5, C=1e30, denom=4.0)
    assert np.array_equal(out.cpu().numpy(), (sums.sum(0) / 8).astype(np.float32))
    assert (np.abs(n.cpu().numpy() - norms / 2) <= 2 * U * norms / 2).all()
    sq = dp.embedding_sqnorms(i, g, V, mask=m).cpu().numpy()
    assert np.array_equal(sq, (sums ** 2).sum((1, 2)))
    # given factors, powers of two; 1 / B of the building block is one product more
    c = 2.0 ** (np.arange(B) % 5 - 2)
    out = dp.embedding_scaled_accumulate(i, g, torch.from_numpy(c.astype(np.float32)).cuda(), V, mask=m)
    want = (c[:, None, None] * sums).sum(0)
    want = want.astype(np.float32) * (np.float32(1) / np.float32(B))
    assert np.array_equal(out.cpu().numpy(), want)
