"""Attention's largest calls: the limits follow the launches.  On the CPU: what is let through ends at the
workspace limit, so nothing is queued."""
import ctypes
import math

import pytest

from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import DPF_BF16, DPF_ERR_UNSUPPORTED, DpfHeads

UNS, MEMORY = DPF_ERR_UNSUPPORTED, 3


@pytest.fixture()
def L():
    lib = _lib.lib()
    assert lib.dpfused_set_option(b"workspace_limit_bytes", 1) == 0
    yield lib
    lib.dpfused_set_option(b"workspace_limit_bytes", 0)


def at(n):
    return (1 << 20) + (n << 46)


def _h(n, B, T, H, D=1):
    return DpfHeads(at(n), DPF_BF16, 0, B, T, H, D, T * H * D, H * D, D)


def ref(x):
    return ctypes.byref(x)


def _calls(L, B, Tq, Tk, Hq, Hkv):
    """Statuses of the forward and the backward call, with segments."""
    q, k = (lambda n: _h(n, B, Tq, Hq)), (lambda n: _h(n, B, Tk, Hkv))
    forward = L.dpfused_attention(ref(q(1)), ref(k(2)), ref(k(3)), None, at(20), 1, math.nan, ref(q(4)), at(21), None)
    backward = L.dpfused_attention_backward(ref(q(5)), ref(q(1)), ref(k(2)), ref(k(3)), ref(q(4)), at(21), None, at(20),
                                            1, math.nan, ref(q(6)), ref(k(7)), ref(k(8)), None)
    return forward, backward


@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv,forward,backward", [
    (64, 1, 65536, 64, 8, MEMORY, MEMORY),            # single tokens of many long sequences
    (512, 1, 1 << 22, 8, 8, MEMORY, UNS),             # their keys' gradients: too many tiles
    (513, 1, 1 << 22, 8, 8, UNS, UNS),                # 2^31 positions
    (1 << 22, 1, 512, 1, 1, MEMORY, UNS),
    (1 << 22, 1, 513, 1, 1, UNS, UNS),
    (1 << 21, 1, 1, 2, 1, MEMORY, MEMORY),
    (1 << 21, 1, 1, 3, 1, UNS, UNS),
    (1 << 22, 32, 32, 1, 1, MEMORY, MEMORY),
    (1 << 22, 33, 33, 1, 1, UNS, UNS),
    (32, 1 << 22, 1 << 22, 1, 1, MEMORY, MEMORY),
    (33, 1 << 22, 1 << 22, 1, 1, UNS, UNS),
    (1, 1, (1 << 22) + 1, 1, 1, UNS, UNS),
    (32, 1, 1 << 22, 4, 1, MEMORY, MEMORY),
    (33, 1, 1 << 22, 4, 1, MEMORY, UNS),
])
def test_limits(L, B, Tq, Tk, Hq, Hkv, forward, backward):
    assert _calls(L, B, Tq, Tk, Hq, Hkv) == (forward, backward)
