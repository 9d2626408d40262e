"""Refusals of the embedding, log-probability and optimizer entry points (CPU: every check runs
before anything is queued), and pins of their oracle against brute force."""
import ctypes
import math

import numpy as np
import pytest

from oracle import language_model as lm
from sample_gradient_clipping_amd import _lib
from sample_gradient_clipping_amd._lib import (DPF_BF16, DPF_ERR_INVALID_ARGUMENT,
                                               DPF_ERR_UNSUPPORTED, DPF_F32, DPF_I32, DPF_I64,
                                               DpfAct, DpfIds)

FAKE = 0x10000   # aligned, never dereferenced: the calls fail first
BAD, UNS = DPF_ERR_INVALID_ARGUMENT, DPF_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _ids(B=2, T=3, data=FAKE, kind=DPF_I64, reserved=0, sb=None):
    return DpfIds(data, kind, reserved, B, T, T if sb is None else sb)


def _act(B=2, T=3, D=8, dtype=DPF_BF16, data=FAKE, reserved=0, sb=None, st=None):
    st = D if st is None else st
    return DpfAct(data, dtype, reserved, B, T, D, T * st if sb is None else sb, st)


def ref(x):
    return None if x is None else ctypes.byref(x)


IDS_CASES = [
    (dict(ids=None), BAD), (dict(ids=_ids(data=None)), BAD), (dict(ids=_ids(kind=2)), UNS),
    (dict(ids=_ids(reserved=1)), UNS), (dict(ids=_ids(B=0)), BAD), (dict(ids=_ids(T=0)), BAD),
    (dict(ids=_ids(sb=2)), BAD), (dict(ids=_ids(data=FAKE + 4)), UNS),
    (dict(ids=_ids(data=FAKE + 2, kind=DPF_I32)), UNS),
]
TABLE_CASES = [
    (dict(V=0), BAD), (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD),
    (dict(V=(1 << 24) + 1), UNS),
]


@pytest.mark.parametrize("case,status", IDS_CASES + TABLE_CASES + [
    (dict(table=None), BAD), (dict(out=None), BAD), (dict(D=0), BAD), (dict(sv=7), BAD),
    (dict(td=5), UNS), (dict(od=-1), UNS), (dict(table=FAKE + 8), UNS), (dict(out=FAKE + 4), UNS),
    (dict(D=(1 << 22) + 1, sv=1 << 23), UNS), (dict(V=1 << 24, D=1 << 10, sv=1 << 10), UNS),
    (dict(ids=_ids(B=1 << 13, T=1 << 13)), UNS),
])
def test_lookup_refusals(L, case, status):
    a = dict(ids=_ids(), table=FAKE, td=DPF_F32, V=10, D=8, sv=8, scale=1.0, od=DPF_F32, out=FAKE)
    a.update(case)
    assert L.dpfused_embedding_lookup(ref(a["ids"]), a["table"], a["td"], a["V"], a["D"], a["sv"],
                                      None, a["scale"], a["od"], a["out"], None) == status
    assert L.dpfused_last_error()


G_CASES = [
    (dict(G=None), BAD), (dict(G=_act(data=None)), BAD), (dict(G=_act(dtype=7)), UNS),
    (dict(G=_act(B=3)), BAD), (dict(G=_act(T=4)), BAD), (dict(G=_act(st=7, sb=21)), BAD),
    (dict(G=_act(data=FAKE + 4)), UNS),
]


@pytest.mark.parametrize("case,status", IDS_CASES + TABLE_CASES + G_CASES + [
    (dict(C=0.0), BAD), (dict(C=math.nan), BAD), (dict(sigma=-1.0), BAD),
    (dict(C=1e30, sigma=1e30), BAD), (dict(denom=0.0), BAD), (dict(denom=math.inf), BAD),
    (dict(acc=2), BAD), (dict(out=None), BAD), (dict(out=FAKE + 8), UNS),
    (dict(ids=_ids(1, 1 << 24), G=_act(1, 1 << 24, 1 << 22), V=2), UNS),
])
def test_embedding_step_refusals(L, case, status):
    a = dict(ids=_ids(), G=_act(), V=10, scale=1.0, C=1.0, sigma=1.0, denom=2.0, acc=0, out=FAKE)
    a.update(case)
    assert L.dpfused_embedding_clip_accumulate(
        ref(a["ids"]), ref(a["G"]), None, a["V"], a["scale"], a["C"], a["sigma"], 0, 0, a["denom"],
        a["acc"], a["out"], None, None) == status


@pytest.mark.parametrize("case,status", IDS_CASES + TABLE_CASES + G_CASES + [(dict(out=None), BAD)])
def test_embedding_building_block_refusals(L, case, status):
    a = dict(ids=_ids(), G=_act(), V=10, scale=1.0, out=FAKE)
    a.update(case)
    assert L.dpfused_embedding_sqnorms(ref(a["ids"]), ref(a["G"]), None, a["V"], a["scale"], a["out"],
                                       0, None) == status
    assert L.dpfused_embedding_scaled_accumulate(ref(a["ids"]), ref(a["G"]), None, a["V"], a["scale"],
                                                 FAKE, 0.0, 0, 0, a["out"], None) == status


def test_embedding_scaled_accumulate_refusals(L):
    f = lambda c=FAKE, std=0.0, out=FAKE: L.dpfused_embedding_scaled_accumulate(  # noqa: E731
        ref(_ids()), ref(_act()), None, 10, 1.0, c, std, 0, 0, out, None)
    assert f(c=None) == BAD and f(std=-1.0) == BAD and f(std=math.nan) == BAD and f(out=FAKE + 4) == UNS


TARGET_CASES = [(dict(y=_ids(B=3)), BAD), (dict(y=_ids(T=4)), BAD), (dict(y=_ids(kind=9)), UNS),
                (dict(y=_ids(sb=1)), BAD)]
LOGIT_CASES = [(dict(z=None), BAD), (dict(z=_act(dtype=3)), UNS), (dict(z=_act(data=FAKE + 2)), UNS),
               (dict(z=_act(1, 1, (1 << 23) + 1), y=None, logp=None), UNS),
               (dict(z=_act(1 << 12, 1 << 12), y=None, logp=None), UNS)]


@pytest.mark.parametrize("case,status", TARGET_CASES + LOGIT_CASES + [
    (dict(k=-1), BAD), (dict(k=33, z=_act(D=64)), BAD), (dict(k=9), BAD),
    (dict(k=2, tl=None), BAD), (dict(k=2, ti=None), BAD), (dict(y=None), BAD),
    (dict(logp=None, ent=None, lse=None), BAD),
])
def test_logprobs_refusals(L, case, status):
    a = dict(z=_act(), y=_ids(), k=0, logp=FAKE, ent=FAKE, lse=FAKE, tl=FAKE, ti=FAKE)
    a.update(case)
    assert L.dpfused_token_logprobs(ref(a["z"]), ref(a["y"]), None, a["k"], a["logp"], a["ent"],
                                    a["lse"], a["tl"], a["ti"], None) == status


FAR = FAKE + (1 << 20)


@pytest.mark.parametrize("case,status", TARGET_CASES + [
    (dict(z=None), BAD), (dict(z=_act(dtype=3)), UNS), (dict(dz=None), BAD),
    (dict(dz=_act(D=9, data=FAR)), BAD), (dict(dz=_act(B=1, data=FAR)), BAD),
    (dict(lse=None), BAD), (dict(dl=None, dh=None), BAD), (dict(y=None), BAD), (dict(ent=None), BAD),
    (dict(dz=_act(data=FAKE, dtype=DPF_F32)), BAD), (dict(dz=_act(data=FAKE + 16)), BAD),
    (dict(dz=_act(data=FAKE, st=16)), BAD),
])
def test_logprobs_gradient_refusals(L, case, status):
    a = dict(z=_act(), y=_ids(), lse=FAKE, ent=FAKE, dl=FAKE, dh=FAKE, dz=_act(data=FAR))
    a.update(case)
    assert L.dpfused_token_logprobs_backward(ref(a["z"]), ref(a["y"]), None, a["lse"], a["ent"],
                                             a["dl"], a["dh"], ref(a["dz"]), None) == status


def test_oracle_embedding_by_brute_force():
    """Against one-hot matrices: g_i = scale * onehot_i^T G_i, masked rows dropped."""
    rng = np.random.default_rng(0)
    B, T, V, D = 3, 7, 5, 4
    ids = rng.integers(-1, V + 1, (B, T))
    G = rng.standard_normal((B, T, D))
    mask = (rng.random((B, T)) < 0.7).astype(np.uint8)
    out, norms, mag = lm.oracle_embedding(ids, G, mask, V, 2.0, 1.5, 0.0, 0, 0, 4.0)
    total = np.zeros((V, D))
    for i in range(B):
        hot = (ids[i][:, None] == np.arange(V)) * mask[i][:, None]
        g = 2.0 * hot.T @ G[i]
        assert abs(np.linalg.norm(g) - norms[i]) < 1e-12
        total += min(1.0, 1.5 / np.linalg.norm(g)) * g
    assert np.abs(out - total / 4.0).max() < 1e-12 and (mag >= np.abs(out) - 1e-12).all()


def test_oracle_logprobs_by_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    z = rng.standard_normal((2, 3, 9)) * 3
    y = rng.integers(0, 9, (2, 3))
    logp, ent, lse, top, ids = lm.oracle_logprobs(z, y, None, 4)
    t = torch.from_numpy(z).requires_grad_()
    ls = torch.log_softmax(t, -1)
    tl = ls.gather(-1, torch.from_numpy(y)[..., None])[..., 0]
    th = -(ls.exp() * ls).sum(-1)
    for a, b in ((logp, tl), (ent, th), (lse, torch.logsumexp(t, -1)), (top, ls.sort(descending=True).values[..., :4])):
        assert np.abs(a - b.detach().numpy()).max() < 1e-12
    assert np.array_equal(ids, np.argsort(-z, -1)[..., :4])
    dl, dh = rng.standard_normal((2, 3)), rng.standard_normal((2, 3))
    (torch.from_numpy(dl) * tl + torch.from_numpy(dh) * th).sum().backward()
    g = lm.oracle_logprobs_grad(z, y, None, lse, ent, dl, dh)
    assert np.abs(g - t.grad.numpy()).max() < 1e-12


NS = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("case,status", [
    (dict(M=None), BAD), (dict(out=None), BAD), (dict(dt=4), UNS), (dict(n=0), BAD), (dict(r=0), BAD),
    (dict(c=0), BAD), (dict(n=65536), UNS), (dict(r=(1 << 17) + 1), UNS), (dict(c=(1 << 17) + 1), UNS),
    (dict(n=1 << 10, r=1 << 12, c=1 << 12), UNS), (dict(steps=0), BAD), (dict(steps=33), BAD),
    (dict(eps=0.0), BAD), (dict(eps=math.nan), BAD), (dict(co=(4.5, 0.0, 0.0)), BAD),
    (dict(co=(2.0, 0.0, 0.0)), BAD), (dict(co=(1.0, math.inf, 0.0)), BAD),
    (dict(co=(3.4445, -4.775, 3.0315)), BAD), (dict(M=FAKE + 4), UNS), (dict(out=FAKE + 8), UNS),
    (dict(out=FAKE + 16), BAD),
])
def test_orthogonalize_refusals(L, case, status):
    a = dict(M=FAKE, dt=DPF_F32, n=1, r=8, c=8, steps=5, co=NS, eps=1e-7, out=FAR)
    a.update(case)
    assert L.dpfused_orthogonalize(a["M"], a["dt"], a["n"], a["r"], a["c"], a["steps"], *a["co"],
                                   a["eps"], a["out"], None) == status


@pytest.mark.parametrize("case,status", [
    (dict(g=None), BAD), (dict(m=None), BAD), (dict(w=None), BAD), (dict(r=0), BAD), (dict(steps=0), BAD),
    (dict(co=(9.0, 0.0, 0.0)), BAD), (dict(eps=-1.0), BAD), (dict(lr=math.nan), BAD),
    (dict(wd=math.inf), BAD), (dict(beta=1.0), BAD), (dict(beta=-0.1), BAD), (dict(scale=math.inf), BAD),
    (dict(g=FAKE + 4), UNS), (dict(m=FAKE), BAD), (dict(w=FAKE + 64), BAD), (dict(w=FAR + 240), BAD),
])
def test_muon_step_refusals(L, case, status):
    a = dict(g=FAKE, m=FAR, w=FAR + (1 << 20), n=1, r=8, c=8, lr=0.1, beta=0.9, wd=0.0, scale=1.0,
             steps=5, co=NS, eps=1e-7)
    a.update(case)
    assert L.dpfused_muon_step(a["g"], a["m"], a["w"], a["n"], a["r"], a["c"], a["lr"], a["beta"], 1,
                               a["wd"], a["scale"], a["steps"], *a["co"], a["eps"], None) == status


def test_oracle_newton_schulz_by_singular_values():
    from oracle import optim
    rng = np.random.default_rng(4)
    for shape in ((6, 9), (9, 6)):
        M = rng.standard_normal(shape)
        u, s, vt = np.linalg.svd(M, full_matrices=False)
        s = s / np.linalg.norm(s)
        for _ in range(4):
            s = NS[0] * s + NS[1] * s ** 3 + NS[2] * s ** 5
        assert np.abs(optim.newton_schulz(M, 4, NS, 1e-7) - (u * s) @ vt).max() < 1e-12
