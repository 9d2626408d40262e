"""The tiled products of the orthogonalised update.

Bar as in tests/test_gpu_ortho.py: four times the error e32 of the same iteration in plain
float32 products, plus 8 u ||X||_F, u = 2^-24.
"""
import numpy as np
import pytest

from oracle import optim
from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
COEFFS = (3.4445, -4.7750, 2.0315)


def _f32(coeffs):
    return tuple(float(np.float32(x)) for x in coeffs)


def _matrix(rng, R, C, kind):
    if kind == "lowrank":
        k = max(1, min(R, C) // 4)
        M = rng.standard_normal((R, k)) @ rng.standard_normal((k, C)) + 1e-2 * rng.standard_normal((R, C))
    else:
        M = rng.standard_normal((R, C))
    return (M * 1e-3).astype(np.float32)


def _bar(M, steps, coeffs, eps=1e-7):
    ref = optim.newton_schulz(M, steps, _f32(coeffs), eps)
    plain = optim.newton_schulz(M, steps, _f32(coeffs), eps, np.float32).astype(np.float64)
    return ref, 4 * np.linalg.norm(plain - ref) + 8 * U * np.linalg.norm(ref)


# c so small that b / 2c is far above A's eigenvalues, of either sign, near nothing, and b^2 / 4c
# far above a; the usual sets beside them.
@pytest.mark.parametrize("coeffs", [(1.5, -0.625, 0.125), (1.5, -0.5, 0.05), (1.5, -0.5, 0.01), (1.5, -0.5, 1e-3),
                                    (1.5, -0.5, 1e-4), (1.5, -0.5, -1e-5), (1.5, -0.5, 2e-6),
                                    (1.5, -0.5, 1e-30), (1.5, -0.5, 1e-42), (0.2, 1.5, -0.7),
                                    (2.0, -1.5, 0.5), (1.875, -1.25, 0.375), COEFFS])
@pytest.mark.parametrize("kind", ["full", "lowrank"])
@pytest.mark.parametrize("shape", [(160, 200), (330, 140)])
def test_every_size_of_the_last_coefficient(shape, kind, coeffs):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    M = _matrix(np.random.default_rng(sum(shape)), *shape, kind)
    for steps in (1, 5):
        out = dp.orthogonalize(torch.from_numpy(M).cuda(), steps=steps, coeffs=coeffs).cpu().numpy()
        ref, bar = _bar(M, steps, coeffs)
        err = np.linalg.norm(out - ref)
        assert err <= bar, (steps, err / bar)


def test_small_last_coefficient_below_eps_and_in_stacks():
    """Matrices kept at another scale, a zero and a NaN among them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(8)
    M = np.stack([_matrix(rng, 150, 190, "full") for _ in range(4)])
    M[1] *= np.float32(1e-27)
    M[2] = 0.0
    M[3, 4, 5] = np.nan
    out = dp.orthogonalize(torch.from_numpy(M).cuda(), coeffs=(1.5, -0.5, 1e-4)).cpu().numpy()
    for k in (0, 1):
        ref, bar = _bar(M[k], 5, (1.5, -0.5, 1e-4))
        assert np.linalg.norm(out[k] - ref) <= bar
    assert np.count_nonzero(out[2]) == 0 and np.isnan(out[3]).all()


def test_update_size_of_zero():
    """scale 0 is a step of size 0, not the default one: the momentum moves, the weight decays."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(11)
    for shape in ((40, 24), (90, 900), (200, 180)):          # one workgroup, strips, tiles
        g, m, w = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda() for _ in range(3))
        m0, w0 = m.clone(), w.clone()
        dp.muon_step(g, m, w, lr=0.5, beta=0.5, weight_decay=0.5, scale=0.0)
        assert torch.equal(w, w0 * 0.75)
        assert torch.equal(m, m0 * 0.5 + g)
        for bad in (-1.0, -1e-30, float("-inf")):
            with pytest.raises(dp.DpfError):
                dp.muon_step(g, m, w, lr=0.5, scale=bad)
        assert torch.equal(w, w0 * 0.75)
