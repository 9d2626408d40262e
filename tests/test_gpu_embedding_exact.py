"""The embedding's norms and sums where float32 is exact, and at the ends of its range.

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-100, -80, -64, -50, 50, 63, 64, 70, 100])
@pytest.mark.parametrize("shape", [(3, 9, 7, 5), (2, 40, 5, 264), (3, 300, 11, 1032)])
def test_norms_over_the_whole_range(shape, power, dtype):
    """Integers times 2^power: their squares leave float32's range, the norms do not."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V, D = shape
    ids, G, mask = make_case(B, T, V, D, "zipf")
    G[1] = 0.0                                             # a sample of zeros
    sums = exact_sums(ids, G, mask, V)
    norms = np.sqrt((sums ** 2).sum((1, 2)))
    i, g, m = _dev(torch, ids, np.ldexp(G, power), mask, dtype)
    C = float(np.ldexp(norms.max() / 4, power))            # clips every sample but the zeros
    out, n = dp.embedding_clip_accumulate(i, g, V, mask=m, C=C, denom=1.0)
    got = np.ldexp(n.cpu().numpy().astype(np.float64), -power)
    assert (np.abs(got - norms) <= 2 * U * norms).all(), (got, norms)
    sq = dp.embedding_sqnorms(i, g, V, mask=m).cpu().numpy()
    assert np.array_equal(np.ldexp(sq, -2 * power), (sums ** 2).sum((1, 2)))
    # the factor: C rounded, the norm's bar, a division; then a product and a sum per sample
    c = np.where(norms > 0, np.minimum(1.0, norms.max() / 4 / np.maximum(norms, 1e-300)), 1.0)
    want = (c[:, None, None] * sums).sum(0)
    L = max(int((mask != 0).sum()), 1)
    err = np.abs(np.ldexp(out.cpu().numpy().astype(np.float64), -power) - want)
    rows = np.zeros((V, D))
    for b in range(B):                                     # sizes of the terms as they are added
        keep = mask[b] != 0
        np.add.at(rows, ids[b][keep], c[b] * np.abs(G[b][keep]).astype(np.float64))
    assert (err <= (L + 6) * U * rows).all()


def test_a_tiny_and_a_huge_column_side_by_side():
    """One column of a sample far below the others, one far above: each counts as it should."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    G = np.zeros((3, 4, 24), np.float32)
    G[0, :, 3] = 2.0 ** -75
    G[1, :, 3], G[1, :, 4] = 2.0 ** -75, 1.0
    G[2, :, 5], G[2, :, 6] = 2.0 ** 65, 2.0 ** -75
    ids = np.zeros((3, 4), np.int64)
    i, g, _ = _dev(torch, ids, G, None, "f32")
    sq = dp.embedding_sqnorms(i, g, 2).cpu().numpy()
    assert np.array_equal(sq, np.array([2.0 ** -146, 16.0, 2.0 ** 134]))
