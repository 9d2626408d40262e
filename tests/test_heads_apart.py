"""Outputs that are parts of one array, with the inputs or each other: what shares no element passes
the overlap checks, what does is refused.  On the CPU: the calls end at a later check (the workspace
limit, or an overlap on purpose), so nothing is queued."""
import ctypes
import math

import pytest

from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import (DPF_BF16, DPF_ERR_INVALID_ARGUMENT, DPF_F32, DpfHeads)

BAD, MEMORY = DPF_ERR_INVALID_ARGUMENT, 3
BASE = 1 << 20


@pytest.fixture()
def L():
    lib = _lib.lib()
    assert lib.dpfused_set_option(b"workspace_limit_bytes", 1) == 0
    yield lib
    lib.dpfused_set_option(b"workspace_limit_bytes", 0)


def _heads(array, first, B, T, H, D, strides, dtype=DPF_BF16):
    """H heads of `array` (arrays are far apart) from element `first` on."""
    size = 2 if dtype == DPF_BF16 else 4
    return DpfHeads(BASE + (array << 40) + first * size, dtype, 0, B, T, H, D, *strides)


def _parts(layout, array, B, T, counts, D, dtype=DPF_BF16):
    """The parts of one array, of counts[i] heads each, as torch's strides describe them."""
    n, out, at = sum(counts), [], 0
    for H in counts:
        if layout == "rows":            # [B, T, n, D]
            first, strides = at * D, (T * n * D, n * D, D)
        elif layout == "samples":       # [B, n, T, D]
            first, strides = at * T * D, (n * T * D, D, T * D)
        elif layout == "swapped":       # [T, B, n, D]
            first, strides = at * D, (n * D, B * n * D, D)
        else:                           # "heads": [B, T, H, parts, D]
            first, strides = len(out) * D, (T * n * D, n * D, len(counts) * D)
        out.append(_heads(array, first, B, T, H, D, strides, dtype))
        at += H
    return out


def ref(x):
    return None if x is None else ctypes.byref(x)


def _moved(x, by):
    return DpfHeads(x.data + by * (2 if x.dtype == DPF_BF16 else 4), x.dtype, 0, x.B, x.T, x.H, x.D, x.stride_b,
                    x.stride_t, x.stride_h)


def _backward(L, dq, dk, dv, inputs=None):
    dout, q, k, v, out = inputs or [_heads(20 + i, 0, t.B, t.T, t.H, t.D, (t.T * t.H * t.D, t.H * t.D, t.D), t.dtype)
                                    for i, t in enumerate((dq, dq, dk, dk, dq))]
    return L.dpfused_attention_backward(ref(dout), ref(q), ref(k), ref(v), ref(out), BASE + (30 << 40), None, None, 1,
                                        math.nan, ref(dq), ref(dk), ref(dv), None)


def _rotary(L, q, k, q_out, k_out):
    return L.dpfused_qk_norm_rotary(ref(q), ref(k), BASE + (30 << 40), BASE + (31 << 40), 1e-6, None, 0, 1.0, 0, None,
                                    None, ref(q_out), ref(k_out), None)


def _rotary_backward(L, gq, gk, q, k, dq, dk):
    w = [BASE + (n << 40) for n in range(30, 34)]
    return L.dpfused_qk_norm_rotary_backward(ref(gq), ref(gk), ref(q), ref(k), w[0], w[1], 1e-6, None, 0, 1.0, 0, None,
                                             None, ref(dq), ref(dk), w[2], w[3], None)


SHAPES = [(1, 1), (2, 1), (16, 1), (1, 2), (2, 2), (5, 7), (3, 50)]
LAYOUTS = ["rows", "samples", "swapped", "heads"]


def _counts(layout):
    return [(4, 4, 4)] if layout == "heads" else [(4, 4, 4), (6, 2, 2), (8, 1, 1), (1, 1, 1)]


@pytest.mark.parametrize("dtype", [DPF_BF16, DPF_F32])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,T", SHAPES)
def test_parts_of_one_array_are_apart(L, B, T, layout, dtype):
    for counts in _counts(layout):
        for D in (8, 45):
            q, k, v = _parts(layout, 1, B, T, counts, D, dtype)
            # gradients as parts of one array
            assert _backward(L, q, k, v) == MEMORY, (counts, D, L.dpfused_last_error())
            # and beside the forward call's tensors, all parts of one
            if layout != "heads":
                six = _parts(layout, 1, B, T, counts + counts, D, dtype)
                other = [_heads(40 + i, 0, B, T, counts[0], D, (T * counts[0] * D, counts[0] * D, D), dtype)
                         for i in range(2)]
                assert _backward(L, *six[3:], inputs=[other[0], *six[:3], other[1]]) == MEMORY
            # the rotation of queries and keys where they are: q_out passes, k_out is refused on purpose
            assert _rotary(L, q, k, q, _moved(k, 1)) == BAD
            assert b"k_out overlaps its input" in L.dpfused_last_error(), L.dpfused_last_error()
            gq, gk, _ = _parts(layout, 2, B, T, counts, D, dtype)
            assert _rotary_backward(L, gq, gk, q, k, gq, gk) == MEMORY, L.dpfused_last_error()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,T", SHAPES)
def test_overlapping_parts_are_refused(L, B, T, layout):
    """Each pair moved together until the first and the last element of one lies in the other."""
    for counts in _counts(layout):
        D = 8
        q, k, v = _parts(layout, 1, B, T, counts, D)
        for by in (1, D - 1, D):
            assert _backward(L, q, _moved(k, -by), _moved(v, D)) == BAD, (counts, by)
            assert _backward(L, q, k, _moved(v, -by)) == BAD, (counts, by)
        assert _backward(L, q, _moved(q, 0) if counts[0] == counts[1] else k, k) == BAD
        gq, gk, _ = _parts(layout, 2, B, T, counts, D)
        assert _rotary_backward(L, gq, _moved(gk, -1), q, k, gq, _moved(gk, -1)) == BAD
        assert _rotary(L, q, k, _moved(q, 1), k) == BAD and b"q_out" in L.dpfused_last_error()


def _elements(t):
    return {t.data // 2 + b * t.stride_b + i * t.stride_t + h * t.stride_h + d for b in range(t.B)
            for i in range(t.T) for h in range(t.H) for d in range(t.D)}


def test_no_shared_element_is_let_through(L):
    """Random strides and offsets: whatever passes shares no element, counted one by one."""
    import random
    rng = random.Random(4)
    passed = 0
    for _ in range(4000):
        B, T, H, D = rng.randint(1, 3), rng.randint(1, 3), rng.choice([1, 2, 4]), rng.randint(1, 4)

        def some(first):
            order, strides, at = rng.sample(range(3), 3), [0, 0, 0], D
            for k in order:
                strides[k] = at + rng.choice([0, 0, D, 2 * D, rng.randint(0, 6)])
                at = strides[k] * (B, T, H)[k]
            return _heads(1, first, B, T, H, D, strides)
        dq, dk = some(0), some(rng.randint(0, 40))
        if rng.random() < 0.5:
            dk = _heads(1, rng.randint(0, 40), B, T, H, D, (dq.stride_b, dq.stride_t, dq.stride_h))
        dv = _heads(2, 0, B, T, H, D, (T * H * D, H * D, D))
        status = _backward(L, dq, dk, dv)
        apart = not (_elements(dq) & _elements(dk))
        assert status == (MEMORY if apart else BAD) or (apart and status == BAD), (status, apart)
        passed += status == MEMORY
    assert passed > 400
