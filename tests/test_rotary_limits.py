"""The rotation's largest calls: a launch holds fewer than 2^32 threads, 256 for each position."""
import ctypes

import pytest

from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import DPF_ERR_UNSUPPORTED, DPF_F32, DpfHeads


def _h(n, B, T, H):
    return DpfHeads((1 << 20) + (n << 44), DPF_F32, 0, B, T, H, 3, T * H * 3, H * 3, 3)


def ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("B,T", [(1 << 24, 1), (1, 1 << 24), (1 << 12, 1 << 12), (3, 5592406)])
def test_as_many_positions_as_threads_allow(B, T):
    lib, at = _lib.lib(), [(1 << 20) + (n << 44) for n in range(10, 15)]
    q, k, a, b, c, d = (_h(n, B, T, H) for n, H in enumerate((5, 1, 5, 1, 5, 1)))
    assert lib.dpfused_qk_norm_rotary(ref(q), ref(k), at[0], at[1], 1e-6, at[2], 1, 1.0, 0, None, None,
                                      ref(a), ref(b), None) == DPF_ERR_UNSUPPORTED
    assert lib.dpfused_qk_norm_rotary_backward(ref(c), ref(d), ref(q), ref(k), at[0], at[1], 1e-6, at[2], 1, 1.0, 0,
                                               None, None, ref(a), ref(b), at[3], at[4], None) == DPF_ERR_UNSUPPORTED
