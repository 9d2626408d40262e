"""That the embedding tests on integers notice one position (CPU: the mistake is planted in the
expected values)."""
import numpy as np
import pytest

from tests.embedding_integers import CASES, exact_sums, make_case

NORM_BAR = 2 * 2.0 ** -24


@pytest.mark.parametrize("case", CASES)
def test_sums_and_squares_are_exact(case):
    ids, G, mask = make_case(*case)
    sums = exact_sums(ids, G, mask, case[2])
    # 8 squares are added in float32, and segments of the whole batch with factors 1/4 .. 4
    assert 8 * (sums ** 2).max() < 2 ** 24
    assert 16 * np.abs(sums).sum(0).max() < 2 ** 24


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("times", [0, 2])
def test_one_position_is_noticed(case, times):
    """Left out or counted twice, first, last or anywhere."""
    B, T, V, D, _ = case
    ids, G, mask = make_case(*case)
    sums = exact_sums(ids, G, mask, V)
    norms = np.sqrt((sums ** 2).sum((1, 2)))
    rng = np.random.default_rng(T)
    for t in {0, T - 1, T // 2, *rng.integers(0, T, 6).tolist()}:
        i = int(rng.integers(B))
        if mask is not None and mask[i, t] == 0:
            continue
        wrong = sums[i].copy()
        wrong[ids[i, t]] += (times - 1) * G[i, t]
        assert (wrong != sums[i]).any()
        n = np.sqrt((wrong ** 2).sum())
        assert abs(n - norms[i]) > 4 * NORM_BAR * norms[i], (i, t)
