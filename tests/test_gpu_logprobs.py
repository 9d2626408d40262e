"""Token log probabilities and their gradient against the fp64 oracle.

Bars, with u = 2^-24 and n = V / 64 + 64 the most additions behind any one term of a
sum (each thread's share of a row, then the joins):
  lse       S is a sum of V positive terms, each with an exponential good to 4 u and an
            argument off by u |d| (d = z - max): rel(S) <= (n + 4 + dbar) u with dbar the
            p-weighted mean of |d|; two roundings at the size of lse
  logp, top_logp   the same and a rounding at the size of z
  entropy   log S as above, and S1 / S: (n + 4 + 2 dmax) u (dbar + 1), dmax the largest
            |d| that still has a weight
  gradient  p off by (|lp| + 6) u; each product one rounding; bf16 outputs are the
            float32 ones rounded, bit for bit
"""
import numpy as np
import pytest

from oracle import dp_linear
from oracle.language_model import oracle_logprobs, oracle_logprobs_grad
from tests.gpu_helpers import need_gpu, to_dev
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _case(rng, B, T, V, dtype, spread=3.0):
    z = (rng.standard_normal((B, T, V)) * spread).astype(np.float32)
    y = rng.integers(0, V, (B, T))
    y.flat[:: 9] = -100
    y.flat[4 :: 13] = V
    return (f32_to_bf16_bits(z) if dtype == "bf16" else z), y


def _bars(z, V):
    m = z.max(-1, keepdims=True)
    d = np.where(np.isfinite(z), m - z, 0.0)
    p = np.where(np.isfinite(z), np.exp(-d), 0.0)
    S = p.sum(-1)
    p /= S[..., None]
    dbar = (p * d).sum(-1)
    dmax = np.minimum(d.max(-1), 104.0)
    n = V / 64 + 64
    lse = np.abs(m[..., 0]) + np.log(S)
    t_lse = U * (n + 4 + dbar + 2 * lse + 2)
    t_ent = t_lse + U * ((n + 4 + 2 * dmax) * (dbar + 1) + 2 * np.log(S) + 2)
    return t_lse, t_ent


def _forward(torch, dp, z, y, mask, dtype, top_k, i32=False):
    r = dp.token_logprobs(to_dev(z, dtype, torch),
                          torch.from_numpy(y).to(torch.int32 if i32 else torch.int64).cuda(),
                          mask=None if mask is None else torch.from_numpy(mask).cuda(), top_k=top_k)
    torch.cuda.synchronize()
    return r


def _check(torch, dp, z, y, mask, dtype, top_k, r):
    B, T, V = z.shape
    w = dp_linear.widen(z, dtype)
    logp, ent, lse, top, ids = oracle_logprobs(w, y, mask, top_k)
    t_lse, t_ent = _bars(w, V)
    big = U * np.abs(w).max(-1)
    for got, want, tol in ((r.lse, lse, t_lse), (r.entropy, ent, t_ent), (r.logp, logp, t_lse + 2 * big)):
        err = np.abs(got.cpu().numpy() - want)
        assert (err <= tol).all(), float((err / tol).max())
    if top_k:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)
        err = np.abs(r.top_logp.cpu().numpy() - top)
        assert (err <= (t_lse + 2 * big)[..., None]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top_k", [0, 1, 5, 32])
@pytest.mark.parametrize("shape", [(1, 1, 33), (2, 5, 100), (3, 7, 1000), (1, 1, 8192), (2, 3, 32000),
                                   (1, 4, 50257), (2, 2, 4097), (1, 2, 131073), (1, 1, 262144)])
def test_matches_oracle(shape, top_k, dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape) + top_k)
    z, y = _case(rng, *shape, dtype)
    mask = None
    if top_k == 5:
        mask = (rng.random(shape[:2]) < 0.6).astype(np.uint8)
    r = _forward(torch, dp, z, y, mask, dtype, top_k, i32=top_k == 1)
    _check(torch, dp, z, y, mask, dtype, top_k, r)


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 257, 511, 2047, 2048, 2049])
def test_short_rows(V):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V)
    for dtype in ("bf16", "f32"):
        z, y = _case(rng, 3, 11, V, dtype)
        k = min(V, 8)
        _check(torch, dp, z, y, None, dtype, k, _forward(torch, dp, z, y, None, dtype, k))


@pytest.mark.parametrize("V", [40, 4097, 50257])
def test_equal_logits_go_to_the_lowest_index(V):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V)
    z = np.zeros((2, 3, V), np.float32)
    z[0, 1] = rng.integers(0, 3, V)
    z[1, 2, V // 2:] = 1.0
    z[1, 1] = -0.0                                     # -0 and +0 are equal
    z[1, 1, ::2] = 0.0
    y = rng.integers(0, V, (2, 3))
    _check(torch, dp, z, y, None, "f32", 32, _forward(torch, dp, z, y, None, "f32", 32))


@pytest.mark.parametrize("top_k", [1, 3, 32])
@pytest.mark.parametrize("V", [700, 4096, 16385, 32769, 70001])
def test_ordered_and_nearly_equal_logits(V, top_k):
    """Alternatives that keep being replaced (rising logits), that come first, that sit in one
    wave's part, and more candidates than a list holds."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V + top_k)
    rise = np.arange(V, dtype=np.float32) / V
    z = np.empty((2, 4, V), np.float32)
    z[0, 0], z[0, 1] = rise, rise[::-1]
    z[0, 2] = np.floor(rise * 40)                      # steps of equal ones, rising
    z[0, 3] = np.floor(rise[::-1] * 40)
    z[1, 0] = rng.integers(0, 50, V)
    z[1, 1] = np.where(np.arange(V) % 512 < 8, 1.0, 0.0) + rng.integers(0, 2, V)
    z[1, 2] = -1e4
    z[1, 2, V // 2: V // 2 + 5] = rng.standard_normal(5)
    z[1, 3] = rng.standard_normal(V)
    y = rng.integers(0, V, (2, 4))
    y[1, 2] = V // 2
    for dtype in ("f32", "bf16"):
        x = f32_to_bf16_bits(z) if dtype == "bf16" else z
        _check(torch, dp, x, y, None, dtype, top_k, _forward(torch, dp, x, y, None, dtype, top_k))


@pytest.mark.parametrize("top_k", [0, 5, 32])
@pytest.mark.parametrize("dtype,V", [("f32", 2049), ("f32", 4001), ("f32", 7000), ("bf16", 4097),
                                     ("bf16", 8003), ("bf16", 12345)])
def test_many_rows(V, dtype, top_k):
    """Rows of two or more chunks by one wave, or by four: where there are many.  The same rows
    over and over (at other alignments, so not bit for bit), in two calls alike."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V + top_k)
    z, y = _case(rng, 4, 75, V, dtype)
    few = _forward(torch, dp, z, y, None, dtype, top_k)                  # 300 rows
    _check(torch, dp, z, y, None, dtype, top_k, few)
    reps = 4200 // 75 + 1
    zs = to_dev(z[:1], dtype, torch).repeat(reps, 1, 1)
    ys = torch.from_numpy(y[:1]).cuda().repeat(reps, 1)
    many, again = (dp.token_logprobs(zs, ys, top_k=top_k) for _ in range(2))
    for a, b in zip(many, again):
        assert a is None or torch.equal(a, b)
    for k in (0, 1, reps // 2, reps - 1):
        part = type(many)(*(None if x is None else x[k:k + 1] for x in many))
        _check(torch, dp, z[:1], y[:1], None, dtype, top_k, part)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [16383, 16384, 32767, 32768, 32776, 65535, 65545])
def test_rows_at_the_edges_of_parts(V, dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V)
    z, y = _case(rng, 1, 3, V, dtype)
    _check(torch, dp, z, y, None, dtype, 8, _forward(torch, dp, z, y, None, dtype, 8))


@pytest.mark.parametrize("V", [50, 4100, 50257])
def test_masked_vocabulary_and_large_logits(V):
    """-inf logits are tokens of probability 0; the type's lowest value and +-1e4 stay finite."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V)
    z, y = _case(rng, 2, 4, V, "f32")
    z[0, 0, rng.random(V) < 0.9] = -np.inf
    z[0, 1, :] = -np.inf
    z[0, 1, V // 3] = 2.0                              # one token left: entropy 0
    z[0, 2] = np.finfo(np.float32).min
    z[0, 3, ::2] = np.finfo(np.float32).min
    z[1, 0] *= 1e4
    z[1, 1] += 3e4
    y[0, 0] = int(np.argmin(z[0, 0]))                  # a target of probability 0
    r = _forward(torch, dp, z, y, None, "f32", 3)
    w = z.astype(np.float64)
    logp, ent, lse, top, ids = oracle_logprobs(w, y, None, 3)
    t_lse, t_ent = _bars(w, V)
    finite = np.where(np.isfinite(w), np.abs(w), 0).max(-1)
    got = r.logp.cpu().numpy()
    assert got[0, 0] == -np.inf and logp[0, 0] == -np.inf
    ok = np.isfinite(logp)
    assert (np.abs(got[ok] - logp[ok]) <= (t_lse + 2 * U * finite)[ok]).all()
    assert (np.abs(r.lse.cpu().numpy() - lse) <= t_lse).all()
    assert (np.abs(r.entropy.cpu().numpy() - ent) <= t_ent).all()
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    assert abs(float(r.entropy[0, 1])) <= 4 * U and abs(float(r.top_logp[0, 1, 0])) <= 4 * U


@pytest.mark.parametrize("V", [50, 8200])
def test_not_a_number(V):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V)
    z, y = _case(rng, 1, 5, V, "f32")
    y[:] = 3
    z[0, 0, 10] = np.nan
    z[0, 1, 10] = np.inf
    z[0, 2] = -np.inf
    z[0, 3] = np.nan
    z[0, 3, 20] = 1.0
    r = _forward(torch, dp, z, y, None, "f32", 4)
    assert torch.isnan(r.logp[0, :4]).all() and torch.isnan(r.entropy[0, :4]).all()
    assert torch.isnan(r.top_logp[0, :4]).all()
    assert torch.isnan(r.lse[0, [0, 1, 3]]).all() and float(r.lse[0, 2]) == -np.inf
    keep = np.where(np.isnan(z[0, 0]), -np.inf, z[0, 0])
    assert r.top_ids[0, 0].tolist() == np.argsort(-keep, kind="stable")[:4].tolist()
    assert int(r.top_ids[0, 1, 0]) == 10
    assert r.top_ids[0, 2].tolist() == [0, 1, 2, 3]
    assert r.top_ids[0, 3].tolist() == [20, -1, -1, -1]
    assert torch.isfinite(r.logp[0, 4]) and torch.isfinite(r.top_logp[0, 4]).all()


def test_masked_rows_are_never_read():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    z = torch.randn(2, 6, 300, device="cuda")
    y = torch.randint(0, 300, (2, 6), device="cuda")
    mask = torch.tensor([[1, 0, 1, 1, 0, 0], [0] * 6], dtype=torch.uint8, device="cuda")
    dirty = torch.where(mask[..., None] != 0, z, torch.full_like(z, float("nan")))
    a, b = (dp.token_logprobs(t, y, mask=mask, top_k=3) for t in (z, dirty))
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert (a.top_ids[mask == 0] == -1).all() and (a.logp[mask == 0] == 0).all()
    g = torch.randn(2, 6, device="cuda")
    bad = torch.where(mask != 0, g, torch.full_like(g, float("nan")))
    p = dp.token_logprobs_backward(z, y, a.lse, g, mask=mask)
    q = dp.token_logprobs_backward(dirty, y, a.lse, bad, mask=mask)
    assert torch.equal(p, q) and torch.count_nonzero(p[mask == 0]) == 0


@pytest.mark.parametrize("ti,to", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 5, 33), (3, 4, 1000), (2, 3, 4097), (1, 2, 50257),
                                   (2, 2, 8192)])
def test_gradient_matches_oracle(shape, terms, ti, to):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V = shape
    rng = np.random.default_rng(sum(shape))
    z, y = _case(rng, B, T, V, ti)
    w = dp_linear.widen(z, ti)
    mask = None if T % 2 else (rng.random((B, T)) < 0.7).astype(np.uint8)
    _, ent, lse, _, _ = oracle_logprobs(w, y, None, 0)
    lse, ent = lse.astype(np.float32), ent.astype(np.float32)
    dl = rng.standard_normal((B, T)).astype(np.float32) if terms != "entropy" else None
    dh = rng.standard_normal((B, T)).astype(np.float32) if terms != "logp" else None
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    call = lambda d: dp.token_logprobs_backward(  # noqa: E731
        to_dev(z, ti, torch), torch.from_numpy(y).cuda(), up(lse), up(dl), entropy=up(ent),
        dentropy=up(dh), mask=up(mask), out_dtype=d)
    out = call(torch.float32)
    if to == "bf16":     # the float32 values, rounded once
        bits = call(torch.bfloat16).view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(bits, f32_to_bf16_bits(out.cpu().numpy()))
    wide = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    ref = oracle_logprobs_grad(w, y, mask, wide(lse), wide(ent), wide(dl), wide(dh))
    lp = w - lse[..., None]
    p = np.exp(lp)
    a1 = 0 if dl is None else np.abs(dl)[..., None] * p
    a2 = 0 if dh is None else np.abs(dh)[..., None] * p * (np.abs(lp) + np.abs(ent)[..., None])
    tol = U * (np.abs(lp) + 10) * (a1 + a2) + 4 * U * np.abs(ref) + 1e-37
    err = np.abs(out.cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())


def test_gradient_is_the_forwards_derivative():
    """Central differences of sum(dlogp logp + dH entropy) in float64 along random directions."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(3)
    z, y = _case(rng, 2, 4, 200, "f32")
    y = np.abs(y) % 200
    dl, dh = (rng.standard_normal((2, 4)).astype(np.float32) for _ in range(2))
    r = _forward(torch, dp, z, y, None, "f32", 0)
    g = dp.token_logprobs_backward(torch.from_numpy(z).cuda(), torch.from_numpy(y).cuda(), r.lse,
                                   torch.from_numpy(dl).cuda(), entropy=r.entropy,
                                   dentropy=torch.from_numpy(dh).cuda()).cpu().numpy().astype(np.float64)

    def f(w):
        logp, ent, _, _, _ = oracle_logprobs(w, y, None, 0)
        return (dl * logp + dh * ent).sum()

    for _ in range(4):
        step = rng.standard_normal(z.shape)
        h = 1e-4
        quotient = (f(z + h * step) - f(z - h * step)) / (2 * h)
        # third derivatives of log-softmax and entropy are O(1) per row: h^2 times a few
        # hundred terms, and float32 rounding of the gradient over 1600 terms
        assert abs(quotient - (g * step).sum()) <= 1e-5 * (1 + np.abs(g * step).sum())


def test_gradient_in_place_and_probabilities_of_zero():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    z = torch.randn(2, 3, 1001, device="cuda")
    z[..., ::3] = float("-inf")
    y = torch.full((2, 3), 4, device="cuda")
    r = dp.token_logprobs(z, y)
    g, h = torch.randn(2, 3, device="cuda"), torch.randn(2, 3, device="cuda")
    ref = dp.token_logprobs_backward(z, y, r.lse, g, entropy=r.entropy, dentropy=h)
    assert torch.isfinite(ref).all() and torch.count_nonzero(ref[..., ::3]) == 0
    same = dp.token_logprobs_backward(z, y, r.lse, g, entropy=r.entropy, dentropy=h, out=z)
    assert same.data_ptr() == z.data_ptr() and torch.equal(ref, z)


@pytest.mark.parametrize("V,extra", [(1000, 24), (1000, 4), (999, 2), (50257, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_logits(dtype, V, extra):
    """logits[:, :-1, :V] of a padded vocabulary, targets ids[:, 1:], the gradient into a slice."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(V + extra)
    z, _ = _case(rng, 3, 6, V + extra, dtype)
    full = to_dev(z, dtype, torch)
    ids = torch.from_numpy(rng.integers(0, V, (3, 6))).cuda()
    part, y = full[:, :-1, :V], ids[:, 1:]
    r = dp.token_logprobs(part, y, top_k=3)
    _check(torch, dp, np.ascontiguousarray(z[:, :-1, :V]), y.cpu().numpy(), None, dtype, 3, r)
    dl = torch.randn(3, 5, device="cuda")
    buf = torch.full_like(full, 7.0)
    dp.token_logprobs_backward(part, y, r.lse, dl, out=buf[:, :-1, :V])
    ref = dp.token_logprobs_backward(part.contiguous(), y.contiguous(), r.lse, dl)
    assert torch.equal(buf[:, :-1, :V], ref)
    assert (buf[:, -1] == 7).all() and (buf[:, :, V:] == 7).all()


def test_without_targets_and_alternatives_alone():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    z = torch.randn(2, 2, 500, device="cuda").bfloat16()
    y = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    a, b = dp.token_logprobs(z, top_k=4), dp.token_logprobs(z, y, top_k=4)
    assert a.logp is None and torch.equal(a.top_ids, b.top_ids) and torch.equal(a.lse, b.lse)
    c = dp.token_logprobs(z, y)
    assert c.top_ids is None and torch.equal(c.logp, b.logp)


@pytest.mark.parametrize("shape", [(1, 1, 32000), (2, 300, 1000), (1, 3, 131072)])
def test_deterministic_on_streams_and_in_graphs(shape):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    z = torch.randn(shape, device="cuda").bfloat16()
    y = torch.randint(0, shape[2], shape[:2], device="cuda")
    ref = dp.token_logprobs(z, y, top_k=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = dp.token_logprobs(z, y, top_k=5)
    s.synchronize()
    for p, q in zip(ref, other):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = dp.token_logprobs(z, y, top_k=5)
    for k in range(4):
        z.copy_(torch.randn(shape, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = dp.token_logprobs(z, y, top_k=5)
        torch.cuda.synchronize()
        for p, q in zip(kept, eager):
            assert torch.equal(p, q)


def test_offsets_past_two_and_four_gib():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    gap = (1 << 31) + 16
    store = torch.zeros(2 * gap + 8192, dtype=torch.bfloat16, device="cuda")
    z = store.as_strided((3, 2, 1000), (gap, 1000, 1))
    small = torch.randn(3, 2, 1000, device="cuda").bfloat16()
    z.copy_(small)
    y = torch.randint(0, 1000, (3, 2), device="cuda")
    a, b = dp.token_logprobs(z, y, top_k=2), dp.token_logprobs(small, y, top_k=2)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    g = torch.randn(3, 2, device="cuda")
    want = dp.token_logprobs_backward(small, y, b.lse, g)
    dp.token_logprobs_backward(z, y, a.lse, g, out=z)
    assert torch.equal(z, want)


def test_binding_refuses_bad_arguments():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    z = torch.zeros(2, 3, 8, device="cuda")
    y = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    f = torch.zeros(2, 3, device="cuda")
    wide = torch.zeros(2, 4, 8, device="cuda")
    for bad in (lambda: dp.token_logprobs(z, y, top_k=9),
                lambda: dp.token_logprobs(z, y, top_k=-1),
                lambda: dp.token_logprobs(z, y[:, :2]),
                lambda: dp.token_logprobs(z, y.float()),
                lambda: dp.token_logprobs(z.half(), y),
                lambda: dp.token_logprobs(z[0], y),
                lambda: dp.token_logprobs(z, y, mask=torch.ones(2, 2, device="cuda", dtype=torch.uint8)),
                lambda: dp.token_logprobs_backward(z, y, f, None),
                lambda: dp.token_logprobs_backward(z, None, f, f),
                lambda: dp.token_logprobs_backward(z, y, f, f, dentropy=f),
                lambda: dp.token_logprobs_backward(z, y, f[:1], f),
                lambda: dp.token_logprobs_backward(z, y, f, f, out=z[:1]),
                lambda: dp.token_logprobs_backward(wide[:, :3], y, f, f, out=wide[:, 1:])):
        with pytest.raises((ValueError, TypeError, dp.DpfError)):
            bad()
