"""Argument checks of the language-model entry points (CPU: they run before anything is queued)."""
import pytest

from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import DPF_ERR_INVALID_ARGUMENT, DPF_ERR_UNSUPPORTED, DPF_F32

FAKE, FAR = 0x10000, 0x10000 + (1 << 20)   # aligned, never dereferenced
BAD, UNS = DPF_ERR_INVALID_ARGUMENT, DPF_ERR_UNSUPPORTED


@pytest.mark.parametrize("coeffs,steps,status", [
    ((1.5, -0.5, 1e-6), 5, UNS), ((1.5, -0.5, 1e-42), 5, UNS), ((1.5, -0.5, -1e-6), 5, UNS),
    ((19.0, -76.0, 60.8), 1, UNS),           # 3.8 times the fifth Chebyshev polynomial
    ((19.0, -76.0, 60.8), 2, BAD), ((4.5, 0.0, 1e-6), 1, BAD),
])
def test_only_growth_refuses_coefficients(coeffs, steps, status):
    """Accepted ones get as far as the misaligned pointer."""
    L = _lib.lib()
    assert L.dpfused_orthogonalize(FAKE + 4, DPF_F32, 1, 8, 8, steps, *coeffs, 1e-7, FAR, None) == status


@pytest.mark.parametrize("scale,status", [(0.0, UNS), (2.0, UNS), (float("nan"), UNS), (-1.0, BAD),
                                          (-1e-30, BAD), (float("-inf"), BAD)])
def test_update_size(scale, status):
    """0 is a size like any other, NaN asks for the default, negative ones are refused."""
    L = _lib.lib()
    assert L.dpfused_muon_step(FAKE + 4, FAR, FAR + (1 << 20), 1, 8, 8, 0.1, 0.9, 1, 0.0, scale, 5,
                               3.4445, -4.775, 2.0315, 1e-7, None) == status


def test_tile_option():
    L = _lib.lib()
    assert L.dpfused_get_option(b"ortho_tile") == 0
    for v in (128, 256, 0):
        assert L.dpfused_set_option(b"ortho_tile", v) == 0
        assert L.dpfused_get_option(b"ortho_tile") == v
    for v in (-1, 1, 64, 512):
        assert L.dpfused_set_option(b"ortho_tile", v) == BAD
    assert L.dpfused_get_option(b"ortho_tile") == 0
