"""Refusals of the attention, rotation and dropout entry points (CPU: every check runs before
anything is queued), and pins of their oracle."""
import ctypes
import math

import numpy as np
import pytest

from oracle import attention as oracle
from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import (DPF_BF16, DPF_ERR_INVALID_ARGUMENT,
                                               DPF_ERR_UNSUPPORTED, DPF_F32, DPF_I64, DpfAct,
                                               DpfHeads, DpfIds)

BASE = 1 << 20
BAD, UNS = DPF_ERR_INVALID_ARGUMENT, DPF_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def at(n):
    """Addresses far apart, never dereferenced: the calls fail first."""
    return BASE + (n << 40)


def _h(n=1, B=2, T=6, H=4, D=8, dtype=DPF_BF16, data=0, reserved=0, sb=None, st=None, sh=None):
    sh = D if sh is None else sh
    st = H * D if st is None else st
    return DpfHeads(None if data is None else at(n) + data, dtype, reserved, B, T, H, D,
                    T * st if sb is None else sb, st, sh)


def ref(x):
    return None if x is None else ctypes.byref(x)


HEADS = [  # what is wrong with one tensor of heads, whichever it is
    (dict(data=None), BAD), (dict(dtype=2), UNS), (dict(reserved=1), UNS), (dict(B=0), BAD),
    (dict(T=0), BAD), (dict(H=0), BAD), (dict(D=0), BAD), (dict(sb=-1), BAD), (dict(st=7), BAD),
    (dict(sh=-8), BAD), (dict(data=1), UNS), (dict(st=1 << 41), UNS), (dict(B=(1 << 30) + 1), UNS),
]
OUT = [(dict(sh=4), BAD), (dict(sb=8), BAD), (dict(st=8), BAD)]   # elements of an output overlap


def _forward(L, q=None, k=None, v=None, out=None, causal=1, scale=math.nan, lse=at(9)):
    t = dict(q=_h(1), k=_h(2), v=_h(3), out=_h(4))
    t.update({n: x for n, x in (("q", q), ("k", k), ("v", v), ("out", out)) if x is not None})
    return L.dpfused_attention(ref(t["q"]), ref(t["k"]), ref(t["v"]), None, None, causal, scale,
                               ref(t["out"]), lse, None)


def _same(**kw):
    return dict(q=_h(1, **kw), k=_h(2, **kw), v=_h(3, **kw), out=_h(4, **kw))


@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
def test_attention_refuses_a_bad_tensor(L, name):
    n = "q k v out".split().index(name) + 1
    for kw, status in HEADS + (OUT if name == "out" else []):
        assert _forward(L, **{name: _h(n, **kw)}) == status, kw
    t = {x: ref(_h(i)) for i, x in enumerate("q k v out".split(), 1)}
    t[name] = None
    assert L.dpfused_attention(t["q"], t["k"], t["v"], None, None, 1, 1.0, t["out"], at(9), None) == BAD


@pytest.mark.parametrize("case,status", [
    (dict(causal=2), BAD), (dict(causal=-1), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=math.inf), BAD), (dict(lse=None), BAD),
    (dict(q=_h(1, dtype=DPF_F32)), UNS), (dict(k=_h(2, dtype=DPF_F32)), UNS), (dict(out=_h(4, dtype=DPF_F32)), UNS),
    (dict(k=_h(2, B=3), v=_h(3, B=3)), BAD), (dict(k=_h(2, D=16), v=_h(3, D=16)), BAD),
    (dict(v=_h(3, T=7)), BAD), (dict(v=_h(3, H=2)), BAD), (dict(q=_h(1, T=7), out=_h(4, T=7)), BAD),
    (dict(k=_h(2, H=3), v=_h(3, H=3)), BAD), (dict(q=_h(1, H=2), out=_h(4, H=2)), BAD),
    (dict(out=_h(4, T=5)), BAD), (dict(out=_h(4, H=8)), BAD), (dict(out=_h(4, D=4)), BAD),
    (_same(D=129), UNS), (_same(T=(1 << 22) + 1, B=1), UNS), (_same(B=1 << 12, T=1 << 12, H=1 << 6), UNS),
    (_same(B=1 << 23, T=1), UNS),
    (dict(out=_h(1)), BAD), (dict(out=_h(2, data=16)), BAD), (dict(out=_h(3, data=-64)), BAD),
])
def test_attention_refusals(L, case, status):
    assert _forward(L, **case) == status
    assert L.dpfused_last_error()


def _part(base, B=2, T=6, heads=12, H=4, first=0, D=8, **kw):
    """Heads first .. first + H of rows of `heads` heads."""
    return _h(base, B=B, T=T, H=H, D=D, st=heads * D, data=first * D * 2, **kw)


def test_attention_overlap_is_seen_by_element(L):
    """Parts of one array's rows pass the overlap check (and go on to a later one)."""
    q, k, v = _part(1, first=0), _part(1, first=4), _part(1, first=8)
    four = dict(q=_part(1, heads=16), k=_part(1, heads=16, first=4), v=_part(1, heads=16, first=8),
                out=_part(1, heads=16, first=12))
    assert _forward(L, **{**four, "out": _part(1, heads=16, first=11)}) == BAD
    assert b"overlaps v" in L.dpfused_last_error()
    assert _forward(L, q=q, k=k, v=v, out=_part(1, first=8)) == BAD
    assert _forward(L, q=q, k=k, v=v, out=_h(1, data=16)) == BAD     # other rows within the range


BWD = "dout q k v out dq dk dv".split()


def _backward(L, lse=at(20), causal=1, scale=math.nan, **kw):
    t = {n: _h(i) for i, n in enumerate(BWD, 1)}
    t.update(kw)
    return L.dpfused_attention_backward(ref(t["dout"]), ref(t["q"]), ref(t["k"]), ref(t["v"]), ref(t["out"]),
                                        lse, None, None, causal, scale, ref(t["dq"]), ref(t["dk"]),
                                        ref(t["dv"]), None)


@pytest.mark.parametrize("name", BWD)
def test_attention_backward_refuses_a_bad_tensor(L, name):
    n = BWD.index(name) + 1
    for kw, status in HEADS + (OUT if name in ("dq", "dk", "dv") else []):
        assert _backward(L, **{name: _h(n, **kw)}) == status, kw
    assert _backward(L, **{name: None}) == BAD
    assert _backward(L, **{name: _h(n, dtype=DPF_F32)}) == UNS
    assert _backward(L, **{name: _h(n, T=5)}) == BAD
    if name in ("dq", "dk", "dv"):
        for other in BWD:
            if other != name:
                assert _backward(L, **{name: _h(BWD.index(other) + 1)}) == BAD, other


def test_attention_backward_refusals(L):
    assert _backward(L, lse=None) == BAD and _backward(L, causal=3) == BAD
    assert _backward(L, scale=-0.5) == BAD
    assert _backward(L, dq=_part(9, first=0), dk=_part(9, first=3), dv=_part(9, first=8)) == BAD


def _rotary(L, q=_h(1), k=_h(2), wq=at(10), wk=at(11), eps=1e-6, freqs=at(12), pairs=4, amplitude=1.0,
            interleaved=0, positions=None, oq=_h(3), ok=_h(4)):
    return L.dpfused_qk_norm_rotary(ref(q), ref(k), wq, wk, eps, freqs, pairs, amplitude, interleaved,
                                    ref(positions), None, ref(oq), ref(ok), None)


def _ids(B=2, T=6, data=at(13), kind=DPF_I64, sb=None):
    return DpfIds(data, kind, 0, B, T, T if sb is None else sb)


ROTARY = [
    (dict(wq=None), BAD), (dict(wk=None), BAD), (dict(eps=0.0), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(eps=math.inf), BAD), (dict(pairs=-1), BAD), (dict(pairs=5), BAD),
    (dict(freqs=None), BAD), (dict(wq=None, wk=None, pairs=0), BAD), (dict(amplitude=math.nan), BAD),
    (dict(amplitude=math.inf), BAD), (dict(interleaved=2), BAD), (dict(freqs=at(12) + 4), UNS),
    (dict(wq=at(10) + 2), UNS), (dict(wk=at(11) + 1), UNS), (dict(positions=_ids(B=3)), BAD),
    (dict(positions=_ids(T=5)), BAD), (dict(positions=_ids(data=None)), BAD),
    (dict(positions=_ids(kind=4)), UNS), (dict(positions=_ids(sb=3)), BAD),
]


@pytest.mark.parametrize("case,status", ROTARY + [
    (dict(q=_h(1, dtype=DPF_F32), oq=_h(3, dtype=DPF_F32)), UNS), (dict(k=_h(2, T=7)), BAD),
    (dict(k=_h(2, D=16)), BAD), (dict(k=_h(2, B=1)), BAD), (dict(oq=_h(3, H=5)), BAD), (dict(ok=_h(4, T=5)), BAD),
    (dict(oq=_h(3, dtype=DPF_F32)), UNS), (dict(oq=None), BAD), (dict(ok=None), BAD), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(oq=_h(1, data=16)), BAD), (dict(oq=_h(2)), BAD), (dict(ok=_h(1)), BAD),
    (dict(ok=_h(3)), BAD), (dict(ok=_h(2, data=-16)), BAD),
    (dict(q=_h(1, D=258), k=_h(2, D=258), oq=_h(3, D=258), ok=_h(4, D=258)), UNS),
    (dict(q=_h(1, B=1 << 12, T=1 << 13), k=_h(2, B=1 << 12, T=1 << 13)), UNS),
] + [(dict(oq=_h(3, **kw)), s) for kw, s in HEADS + OUT] + [(dict(q=_h(1, **kw)), s) for kw, s in HEADS])
def test_rotary_refusals(L, case, status):
    assert _rotary(L, **case) == status


@pytest.mark.parametrize("case,status", ROTARY + [
    (dict(dwq=None), BAD), (dict(dwk=None), BAD), (dict(wq=None, wk=None), BAD), (dict(dwq=at(14) + 2), UNS),
    (dict(gq=None), BAD), (dict(gk=_h(6, H=3)), BAD), (dict(gq=_h(5, T=5)), BAD), (dict(oq=_h(3, H=5)), BAD),
    (dict(gk=_h(6, dtype=DPF_F32)), UNS), (dict(oq=_h(1)), BAD), (dict(oq=_h(6)), BAD), (dict(ok=_h(2)), BAD),
    (dict(ok=_h(5)), BAD), (dict(oq=_h(5, data=16)), BAD), (dict(ok=_h(3)), BAD),
] + [(dict(ok=_h(4, **kw)), s) for kw, s in HEADS + OUT] + [(dict(gq=_h(5, **kw)), s) for kw, s in HEADS])
def test_rotary_backward_refusals(L, case, status):
    a = dict(gq=_h(5), gk=_h(6), q=_h(1), k=_h(2), wq=at(10), wk=at(11), eps=1e-6, freqs=at(12), pairs=4,
             amplitude=1.0, interleaved=0, positions=None, oq=_h(3), ok=_h(4), dwq=at(14), dwk=at(15))
    a.update(case)
    assert L.dpfused_qk_norm_rotary_backward(
        ref(a["gq"]), ref(a["gk"]), ref(a["q"]), ref(a["k"]), a["wq"], a["wk"], a["eps"], a["freqs"], a["pairs"],
        a["amplitude"], a["interleaved"], ref(a["positions"]), None, ref(a["oq"]), ref(a["ok"]), a["dwq"],
        a["dwk"], None) == status


def _act(n=1, B=2, T=3, D=8, dtype=DPF_BF16, data=0, reserved=0, sb=None, st=None):
    st = D if st is None else st
    return DpfAct(None if data is None else at(n) + data, dtype, reserved, B, T, D, T * st if sb is None else sb, st)


@pytest.mark.parametrize("case,status", [
    (dict(x=None), BAD), (dict(y=None), BAD), (dict(p=-0.1), BAD), (dict(p=1.0), BAD), (dict(p=math.nan), BAD),
    (dict(p=1.0 - 2.0 ** -18), BAD), (dict(y=_act(3, D=7)), BAD), (dict(y=_act(3, T=4)), BAD),
    (dict(r=_act(2, B=1)), BAD), (dict(r=_act(2, dtype=DPF_F32)), UNS), (dict(y=_act(3, dtype=DPF_F32)), UNS),
    (dict(y=_act(1, data=16)), BAD), (dict(r=_act(2), y=_act(2, st=16)), BAD),
    (dict(x=_act(1, B=1 << 12, T=1 << 12, D=1 << 11), y=_act(3, B=1 << 12, T=1 << 12, D=1 << 11)), UNS),
] + [(dict(**{t: _act(i, **kw)}), s) for i, t in ((1, "x"), (2, "r"), (3, "y")) for kw, s in (
    (dict(data=None), BAD), (dict(dtype=5), UNS), (dict(reserved=2), UNS), (dict(B=0), BAD), (dict(T=0), BAD),
    (dict(D=0), BAD), (dict(st=7), BAD), (dict(sb=8), BAD), (dict(data=1), UNS))])
def test_dropout_refusals(L, case, status):
    a = dict(x=_act(1), r=None, p=0.1, y=_act(3))
    a.update(case)
    assert L.dpfused_dropout(ref(a["x"]), ref(a["r"]), None, a["p"], 0, 0, ref(a["y"]), None) == status


def test_dropout_blocks(L):
    import sample_gradient_clipping_amd as dp
    assert [dp.dropout_blocks(n) for n in (-1, 0, 1, 8, 9, 1 << 40)] == [0, 0, 1, 1, 2, 1 << 37]


def test_binding_checks_its_arguments():
    torch = pytest.importorskip("torch")
    import sample_gradient_clipping_amd as dp
    x = torch.zeros(2, 3, 4, 8)
    for f in (lambda: dp.attention(x, x, x), lambda: dp.qk_norm_rotary(x, x, freqs=torch.zeros(4)),
              lambda: dp.attention(x[0], x, x), lambda: dp.dropout(x[0], 0.1), lambda: dp.dropout(x, 0.1)):
        with pytest.raises(ValueError):
            f()


def test_rotary_frequencies():
    import sample_gradient_clipping_amd as dp
    plain, one = dp.rotary_frequencies(64, 10000.0, device="cpu")
    j = np.arange(32)
    assert one == 1.0 and np.abs(plain.numpy() / 10000.0 ** (-j / 32) - 1).max() < 1e-14
    lin, _ = dp.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert np.abs(lin.numpy() * 4 / plain.numpy() - 1).max() < 1e-14
    ntk, _ = dp.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1] * 4 / plain[-1]) - 1) < 1e-12
    yarn, size = dp.rotary_frequencies(64, scaling="yarn", factor=4.0, length=2048, device="cpu")
    assert size == 0.1 * math.log(4.0) + 1.0
    turns = 2048 * plain.numpy() / (2 * math.pi)
    ratio = plain.numpy() / yarn.numpy()
    assert np.abs(ratio[turns > 40] - 1).max() < 1e-14 and np.abs(ratio[turns < 0.7] - 4).max() < 1e-12
    assert (np.diff(ratio) >= -1e-12).all() and ((ratio > 1) & (ratio < 3.99)).any()
    for kw in (dict(dim=3), dict(dim=0), dict(dim=8, base=1.0), dict(dim=8, factor=0.5), dict(dim=8, scaling="x"),
               dict(dim=8, scaling="yarn", factor=2.0), dict(dim=8, scaling="yarn", length=9, beta=(1.0, 2.0))):
        with pytest.raises(ValueError):
            dp.rotary_frequencies(**{"device": "cpu", **kw})


# ---------------------------------------------------------------------------
# Pins of the oracle
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("causal", [False, True])
def test_oracle_attention_by_torch_and_differences(causal):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    B, Tq, Tk, Hq, Hkv, D = 2, 5, 7, 4, 2, 3
    q, k, v = (rng.standard_normal(s) for s in ((B, Tq, Hq, D), (B, Tk, Hkv, D), (B, Tk, Hkv, D)))
    dout = rng.standard_normal(q.shape)
    mask = np.ones((B, Tk), np.uint8)
    mask[0, 3] = mask[1, 6] = mask[1, 0] = 0
    seg = np.array([[0, 0, 0, 1, 1, 1, 1], [2, 2, 2, 2, 2, 2, 2]], np.int32)
    (out, _), (lse, _), (dq, _), (dk, _), (dv, _) = oracle.oracle_attention(q, k, v, mask, seg, causal, 0.6, "f32", dout)
    tq, tk, tv = (torch.from_numpy(x).requires_grad_() for x in (q, k, v))
    z = torch.einsum("bihd,bjhd->bhij", tq, tk.repeat_interleave(2, 2)) * 0.6
    ok = torch.from_numpy(np.stack([oracle.allowed(b, Tq, Tk, mask, seg, causal) for b in range(B)]))[:, None]
    live = ok.any(-1, keepdim=True)
    P = torch.softmax(z.masked_fill(~ok & live, -math.inf), -1) * live
    o = torch.einsum("bhij,bjhd->bihd", P, tv.repeat_interleave(2, 2))
    want = torch.autograd.grad(o, (tq, tk, tv), torch.from_numpy(dout))
    assert np.abs(out - o.detach().numpy()).max() < 1e-13 and not out[1, 4].any() and not lse[1, :, 4].any()
    for got, w in zip((dq, dk, dv), want):
        assert np.abs(got - w.numpy()).max() < 1e-13
    # a gradient by differences
    f = lambda x: (oracle.oracle_attention(q, x, v, mask, seg, causal, 0.6, "f32")[0][0] * dout).sum()  # noqa: E731
    for at_ in ((0, 1, 0, 2), (1, 3, 1, 0)):
        e = np.zeros_like(k)
        e[at_] = 1e-5
        assert abs((f(k + e) - f(k - e)) / 2e-5 - dk[at_]) < 1e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotary_by_differences_and_inverse(interleaved):
    rng = np.random.default_rng(5)
    x, w, dy = rng.standard_normal((2, 3, 2, 7)), 1 + rng.standard_normal(7) * 0.2, rng.standard_normal((2, 3, 2, 7))
    freqs, pos = np.array([1.0, 0.1, 0.013]), rng.integers(-5, 900, (2, 3))
    mask = np.array([[1, 0, 1], [1, 1, 1]], np.uint8)
    f = lambda x, w: oracle.oracle_rotary(x, w, 1e-3, freqs, pos, 1.3, interleaved, mask)[0]  # noqa: E731
    dx, _, gw, _ = oracle.oracle_rotary(x, w, 1e-3, freqs, pos, 1.3, interleaved, mask, dy=dy)
    for at_ in ((0, 0, 1, 2), (1, 2, 0, 6), (0, 1, 0, 0)):
        e = np.zeros_like(x)
        e[at_] = 1e-5
        assert abs(((f(x + e, w) - f(x - e, w)) * dy).sum() / 2e-5 - dx[at_]) < 1e-8
    e = np.zeros_like(w)
    e[4] = 1e-5
    assert np.abs(((f(x, w + e) - f(x, w - e)) * dy).sum((1, 2, 3)) / 2e-5 - gw[:, 4]).max() < 1e-8
    y = oracle.oracle_rotary(x, None, 1.0, freqs, pos, 1.0, interleaved, None)[0]
    back = oracle.oracle_rotary(x, None, 1.0, freqs, pos, 1.0, interleaved, None, dy=y)[0]
    assert np.abs(back - x).max() < 1e-13
    # a rotation by pi / 2 takes (a, b) to (-b, a)
    y = oracle.oracle_rotary(np.array([[[[3.0, 4.0]]]]), None, 1.0, [math.pi / 2], np.array([[1]]), 1.0, interleaved, None)[0]
    assert np.abs(y - [-4.0, 3.0]).max() < 1e-15


def test_oracle_dropout_law():
    bits = oracle.dropout_bits(7, 3, 4096)
    assert (bits >= 0).all() and (bits < 65536).all() and abs(bits.mean() / 32767.5 - 1) < 0.05
    assert np.array_equal(oracle.dropout_bits(7, 4, 24), bits[8:32])      # blocks advance by 8 entries
    from oracle.philox import philox_words_scalar
    noise = np.array(philox_words_scalar(7, 3, 2), np.uint32).view(np.uint16)
    assert not np.array_equal(noise.reshape(-1), bits[:16])               # apart from the noise's


@pytest.mark.parametrize("scale", [2.0 ** -65, 1e-38, 2.0 ** 65, 3e38])
def test_scale_out_of_range(scale):
    """lse / scale has to stay finite."""
    L = _lib.lib()
    assert _forward(L, scale=scale) == BAD
    assert _backward(L, scale=scale) == BAD


def test_misaligned_statistics():
    L = _lib.lib()
    for wrong in (1, 2, 3):
        assert _forward(L, lse=at(9) + wrong) == UNS
        assert _backward(L, lse=at(20) + wrong) == UNS
