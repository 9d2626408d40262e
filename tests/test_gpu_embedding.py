"""Embedding lookup and its per-sample clipped gradient against the fp64 oracle.

Bars, with u = 2^-24 (float32 rounding):
  lookup     one float32 product and one rounding: equal bit for bit
  gradient   a float32 sum of L terms is off by at most (L + 2) u times the sum of
             their sizes; the clip factor, scale and 1/denom add four roundings more
             and the factor carries the norm's error; the noise term is held to
             1e-5 sigma C / denom, as the linears' (float32 log, sin and cos)
  norms      of sums off by at most (L + 2) u |g|_abs: the same, relative to the
             norm of the summed sizes
"""
import numpy as np
import pytest

from oracle import dp_linear
from oracle.language_model import active_positions, oracle_embedding
from tests.gpu_helpers import need_gpu, to_dev
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _case(rng, B, T, V, D, dtype, ids="zipf", g_scale=1e-2):
    if ids == "one":
        tok = np.full((B, T), V - 1)
    elif ids == "wild":     # outside [0, V) too, at the limits of the type as well
        tok = rng.integers(-2, V + 3, (B, T))
        tok.flat[:: 7] = np.iinfo(np.int32).max
        tok.flat[3 :: 11] = np.iinfo(np.int32).min
    else:
        tok = np.minimum((np.exp(rng.random((B, T)) * np.log(V + 1.0)) - 1).astype(np.int64), V - 1)
    G = (rng.standard_normal((B, T, D)) * g_scale).astype(np.float32)
    G *= np.exp(rng.standard_normal((B, 1, 1))).astype(np.float32)
    return tok.astype(np.int64), f32_to_bf16_bits(G) if dtype == "bf16" else G


def _mask(rng, B, T, kind):
    if kind is None:
        return None
    if kind == "prefix":
        return (np.arange(T)[None, :] < rng.integers(1, T + 1, (B, 1))).astype(np.uint8)
    m = (rng.random((B, T)) < 0.5).astype(np.uint8) * 3   # any byte but 0 is active
    m[0] = 0                                             # a sample without a token
    return m


def _check(torch, dp, tok, G, V, dtype, mask, scale, C, sigma, seed=5, offset=9, denom=None,
           base=None, dev=None, **kw):
    B, T, D = G.shape
    denom = float(B) if denom is None else denom
    it = torch.int32 if kw.pop("i32", False) else torch.int64
    ids, g, m = dev if dev is not None else (
        torch.from_numpy(tok).to(it).cuda(), to_dev(G, dtype, torch),
        None if mask is None else torch.from_numpy(mask).cuda())
    args = dict(mask=m, scale=scale, C=C, sigma=sigma, seed=seed, offset=offset, denom=denom)
    if base is not None:
        args.update(grad_out=torch.from_numpy(base).cuda(), accumulate=True)
    out, norms = dp.embedding_clip_accumulate(ids, g, V, **args, **kw)
    torch.cuda.synchronize()
    wide = dp_linear.widen(G, dtype)
    ref, rn, mag = oracle_embedding(tok, wide, mask, V, scale, C, sigma, seed, offset, denom)
    act = active_positions(tok, mask, V)
    counts = np.bincount(tok[act], minlength=V) if act.any() else np.zeros(V, int)
    L = max(1, int(counts.max()))
    flat = np.array([np.sqrt(sum((np.abs(scale * wide[i, t])[None] ** 2).sum() for t in range(T)
                                 if act[i, t])) for i in range(B)])
    # |sum| <= the sizes' sum: its norm is at most sqrt(L) times the norm of all rows
    n_tol = (L + 4) * U * np.sqrt(L) * flat + U * rn
    n_err = np.abs(norms.cpu().numpy() - rn)
    assert (n_err <= n_tol).all(), (n_err, n_tol)
    rel_c = np.max(np.where(rn > 0, n_tol / np.maximum(rn, 1e-300), 0.0)) + U
    got = out.cpu().numpy().astype(np.float64)
    tol = ((L + 8) * U + rel_c) * mag + 2 * U * np.abs(ref) + 1e-5 * sigma * C / denom
    if base is not None:
        ref = ref + base
        tol = tol + 2 * U * np.abs(base)
    assert got.shape == ref.shape
    assert (np.abs(got - ref) <= tol + 1e-40).all(), float(np.max(np.abs(got - ref) / (tol + 1e-40)))
    return out, norms


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [None, "prefix", "holes"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (1, 1, 2, 8), (4, 33, 1001, 99), (3, 70, 50, 64),
                                   (5, 130, 600, 132), (2, 300, 4000, 1032), (7, 19, 3, 1100),
                                   (1, 257, 300, 2050)])
def test_gradient_matches_oracle(shape, mask, dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V, D = shape
    rng = np.random.default_rng(sum(shape))
    tok, G = _case(rng, B, T, V, D, dtype)
    m = _mask(rng, B, T, mask)
    C = 1e-2 * np.sqrt(T * D)                       # clips some samples
    _check(torch, dp, tok, G, V, dtype, m, 1.5, C, 0.7, i32=B % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [63, 64, 65, 128, 700, 2049])
def test_one_token_everywhere(T, dtype):
    """Every position is the same token: one run per sample, one segment over all of them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(T)
    tok, G = _case(rng, 3, T, 17, 72, dtype, ids="one")
    out, _ = _check(torch, dp, tok, G, 17, dtype, None, 1.0, 0.5, 0.0)
    assert torch.count_nonzero(out[:16]) == 0


def test_many_sort_chunks_and_digits():
    """More positions than one sort chunk per workgroup holds, ids over three digits."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(3)
    B, T, V, D = 130, 2100, 600000, 4
    tok = rng.integers(0, V, (B, T))
    tok[:, ::3] = rng.integers(0, 40, tok[:, ::3].shape)   # some rows with many positions
    G = rng.standard_normal((B, T, D)).astype(np.float32)
    ids, g = torch.from_numpy(tok).cuda(), torch.from_numpy(G).cuda()
    out = dp.embedding_scaled_accumulate(ids, g, torch.ones(B, device="cuda"), V)
    ref = np.zeros((V, D))
    np.add.at(ref, tok.reshape(-1), G.reshape(-1, D).astype(np.float64))
    mag = np.zeros((V, D))
    np.add.at(mag, tok.reshape(-1), np.abs(G.reshape(-1, D)).astype(np.float64))
    L = np.bincount(tok.reshape(-1), minlength=V)[:, None]
    err = np.abs(out.cpu().numpy() * float(B) - ref)
    assert (err <= (L + 6) * U * mag + 4 * U * np.abs(ref)).all()
    sq = dp.embedding_sqnorms(ids[:3], g[:3], V)
    for i in range(3):
        gi = np.zeros((V, D))
        np.add.at(gi, tok[i], G[i].astype(np.float64))
        assert abs(float(sq[i]) / (gi * gi).sum() - 1) <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ids_outside_the_table_are_inactive(dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(8)
    tok, G = _case(rng, 4, 90, 37, 40, dtype, ids="wild")
    for i32 in (True, False):
        _check(torch, dp, tok, G, 37, dtype, None, 1.0, 0.3, 0.5, i32=i32)
    big = tok.copy()
    big[big < 0] = np.iinfo(np.int64).min
    big[big >= 37] = 1 << 32                     # 0 if it were cut to 32 bits
    ids, g = torch.from_numpy(big).cuda(), to_dev(G, dtype, torch)
    _check(torch, dp, big, G, 37, dtype, None, 1.0, 0.3, 0.0, dev=(ids, g, None))


def test_every_position_inactive_gives_noise_alone():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    ids = torch.full((3, 50), -100, device="cuda")
    G = torch.full((3, 50, 24), float("nan"), device="cuda")
    out, norms = dp.embedding_clip_accumulate(ids, G, 11, C=2.0, sigma=0.5, seed=3, offset=1)
    want = dp.gaussian_fill(3, 1, 11 * 24, scale=1.0) * (0.5 * 2.0) / 3
    assert torch.count_nonzero(norms) == 0
    # one product and one division, against the division as a product with 1/3
    assert torch.allclose(out.reshape(-1), want, rtol=4 * U, atol=0)


def test_masked_rows_are_never_read_and_active_nan_reaches_its_rows():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(2)
    tok, G = _case(rng, 3, 40, 30, 32, "f32")
    m = _mask(rng, 3, 40, "holes")
    ids, mk = torch.from_numpy(tok).cuda(), torch.from_numpy(m).cuda()
    clean = torch.from_numpy(G).cuda()
    dirty = torch.where(mk[..., None] != 0, clean, torch.full_like(clean, float("nan")))
    a, an = dp.embedding_clip_accumulate(ids, clean, 30, mask=mk, C=0.1, sigma=0.5)
    b, bn = dp.embedding_clip_accumulate(ids, dirty, 30, mask=mk, C=0.1, sigma=0.5)
    assert torch.equal(a, b) and torch.equal(an, bn)
    t = int(np.nonzero(m[1])[0][0])
    dirty[1, t, 5] = float("nan")
    c, cn = dp.embedding_clip_accumulate(ids, dirty, 30, mask=mk, C=0.1, sigma=0.0)
    assert torch.isnan(cn[1]) and not torch.isnan(cn[0]) and not torch.isnan(cn[2])
    used = torch.zeros(30, dtype=torch.bool, device="cuda")
    used[ids[1][mk[1] != 0]] = True
    assert torch.isnan(c[used]).all() and not torch.isnan(c[~used]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_ids_and_gradients(dtype):
    """ids[:, 1:] of a longer array, G a slice of wider rows and of longer samples."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(6)
    B, T, V, D = 3, 61, 90, 40
    for extra in (8, 4, 3):
        tok, _ = _case(rng, B, T + 1, V, D, dtype)
        _, G = _case(rng, B, T + 5, V, D + extra, dtype)
        ids = torch.from_numpy(tok).cuda()[:, 1:]
        g = to_dev(G, dtype, torch)[:, :T, :D]
        _check(torch, dp, tok[:, 1:], G[:, :T, :D], V, dtype, None, 1.0, 0.2, 0.3,
               dev=(ids, g, None))


@pytest.mark.parametrize("D", [64, 37])
def test_micro_batches_add_up(D):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(D)
    tok, G = _case(rng, 4, 50, 120, D, "bf16")
    base = rng.standard_normal((120, D)).astype(np.float32)
    _check(torch, dp, tok, G, 120, "bf16", None, 1.0, 0.2, 0.9, denom=16.0, base=base)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [4, 97, 1282, 1300, 2564])
def test_long_segments_in_several_column_groups(D, dtype):
    """Few tokens, many positions: most of a row's positions come in whole blocks."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(D)
    tok, G = _case(rng, 5, 131, 4, D, dtype)
    base = rng.standard_normal((9, D)).astype(np.float32)
    for m, sigma in (("holes", 0.0), ("prefix", 0.6)):
        _check(torch, dp, tok, G, 9, dtype, _mask(rng, 5, 131, m), 1.0, 0.3, sigma, denom=7.0, base=base)


@pytest.mark.parametrize("D", [8, 13])
@pytest.mark.parametrize("T", [10, 400])
def test_accumulating_without_noise_leaves_other_rows(T, D):
    """Rows that no active position adds to keep their bits, NaN and -0 among them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(T)
    tok, G = _case(rng, 2, T, 20, D, "f32")
    tok[tok == 7] = 8
    base = rng.standard_normal((30, D)).astype(np.float32)
    base[7], base[25], base[26] = -0.0, np.nan, np.inf
    out = torch.from_numpy(base).cuda()
    dp.embedding_clip_accumulate(torch.from_numpy(tok).cuda(), to_dev(G, "f32", torch), 30, C=1.0,
                                 grad_out=out, accumulate=True)
    got = out.cpu().numpy()
    rest = np.setdiff1d(np.arange(30), tok)
    assert {7, 25, 26} <= set(rest)
    assert np.array_equal(got[rest].view(np.uint32), base[rest].view(np.uint32))
    assert (got[np.unique(tok)] != base[np.unique(tok)]).any(axis=1).all()


def test_group_clipping_with_a_linear_layer():
    """One factor per sample over the embedding and a linear, from the building blocks."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(12)
    B, T, V, D, dout = 3, 40, 70, 32, 24
    tok, G = _case(rng, B, T, V, D, "f32")
    X = rng.standard_normal((B, T, D)).astype(np.float32)
    H = (rng.standard_normal((B, T, dout)) * 1e-2).astype(np.float32)
    ids, g, x, h = (torch.from_numpy(a).cuda() for a in (tok, G, X, H))
    sq = dp.embedding_sqnorms(ids, g, V, scale=2.0)
    dp.per_sample_sqnorms(x, h, out=sq, accumulate=True)
    _, en, _ = oracle_embedding(tok, G.astype(np.float64), None, V, 2.0, 1.0, 0.0, 0, 0, 1.0)
    ln = np.array([np.linalg.norm(H[i].astype(np.float64).T @ X[i]) for i in range(B)])
    want = en ** 2 + ln ** 2
    assert np.abs(sq.cpu().numpy() / want - 1).max() <= 1e-5
    C = float(np.sqrt(np.median(want)))
    c, _ = dp.clip_factors(sq, C)
    out = dp.embedding_scaled_accumulate(ids, g, c, V, scale=2.0, noise_std=0.3, seed=2, offset=4)
    ref = np.zeros((V, D))
    for i in range(B):
        np.add.at(ref, tok[i], 2.0 * min(1.0, C / np.sqrt(want[i])) * G[i].astype(np.float64))
    from oracle.philox import gaussian
    ref = (ref + 0.3 * gaussian(2, 4, V * D).reshape(V, D)) / B
    assert np.abs(out.cpu().numpy() - ref).max() <= 1e-5 * (np.abs(ref).max() + 0.3)


def test_gradient_is_the_lookups_derivative():
    """Central differences of <lookup(table), G> along a direction: the function is linear in the
    table, so the quotient has only rounding; the gradient is one sample's, unclipped."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(21)
    T, V, D, scale = 80, 45, 36, 3.0
    tok, G = _case(rng, 1, T, V, D, "f32", g_scale=1.0)
    ids, g = torch.from_numpy(tok).cuda(), torch.from_numpy(G).cuda()
    grad, _ = dp.embedding_clip_accumulate(ids, g, V, scale=scale, C=1e30, sigma=0.0)
    table = torch.randn(V, D, device="cuda")
    step = torch.randn(V, D, device="cuda")
    h = 0.25
    f = lambda w: float((dp.embedding_lookup(ids, w, scale=scale).double() * g.double()).sum())
    quotient = (f(table + h * step) - f(table - h * step)) / (2 * h)
    slope = float((grad.double() * step.double()).sum())
    # every entry of the two tables is off by u relative, summed over T D terms in quadrature
    noise = 4 * U * scale * float(g.abs().max()) * float(table.abs().max()) * np.sqrt(T * D) / h * 8
    assert abs(quotient - slope) <= noise


def test_same_result_on_other_streams_and_in_graphs():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(31)
    tok, G = _case(rng, 4, 600, 500, 136, "bf16")
    ids, g = torch.from_numpy(tok).cuda(), to_dev(G, "bf16", torch)
    ref, rn = dp.embedding_clip_accumulate(ids, g, 500, C=0.1, sigma=1.0, seed=4)
    for _ in range(3):
        again, an = dp.embedding_clip_accumulate(ids, g, 500, C=0.1, sigma=1.0, seed=4)
        assert torch.equal(ref, again) and torch.equal(rn, an)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, on = dp.embedding_clip_accumulate(ids, g, 500, C=0.1, sigma=1.0, seed=4)
    s.synchronize()
    assert torch.equal(ref, other) and torch.equal(rn, on)
    out, norms = torch.zeros_like(ref), torch.zeros_like(rn)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.embedding_clip_accumulate(ids, g, 500, C=0.1, sigma=1.0, seed=4, grad_out=out,
                                     norms_out=norms)
    for k in range(4):
        ids.copy_(torch.from_numpy((tok + k) % 500))
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager, en = dp.embedding_clip_accumulate(ids, g, 500, C=0.1, sigma=1.0, seed=4)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(norms, en)


def test_outputs_stay_inside_their_buffers():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(41)
    for V, D in ((7, 36), (13, 5), (50, 1028)):
        tok, G = _case(rng, 2, 33, V, D, "f32")
        buf = torch.full((V * D + 512,), 7.0, device="cuda")
        out = buf[256:256 + V * D].view(V, D)
        dp.embedding_clip_accumulate(torch.from_numpy(tok).cuda(), torch.from_numpy(G).cuda(), V,
                                     C=1.0, sigma=1.0, grad_out=out)
        rows = torch.full((2 * 33 * D + 512,), 7.0, device="cuda")
        look = rows[256:256 + 2 * 33 * D].view(2, 33, D)
        dp.embedding_lookup(torch.from_numpy(tok).cuda(), out, out=look)
        torch.cuda.synchronize()
        for b, n in ((buf, V * D), (rows, 2 * 33 * D)):
            assert (b[:256] == 7).all() and (b[256 + n:] == 7).all()


@pytest.mark.parametrize("ti", ["bf16", "f32"])
@pytest.mark.parametrize("to", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (3, 17, 29, 7), (2, 65, 40, 36), (4, 9, 100, 520),
                                   (1, 300, 11, 2048), (16, 1, 64, 768)])
def test_lookup_is_exact(shape, to, ti):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, T, V, D = shape
    rng = np.random.default_rng(sum(shape))
    tok, _ = _case(rng, B, T, V, 1, "f32", ids="wild" if T > 2 else "zipf")
    table = rng.standard_normal((V, D)).astype(np.float32)
    stored = f32_to_bf16_bits(table) if ti == "bf16" else table
    exact = bf16_bits_to_f32(stored) if ti == "bf16" else stored
    for mask, scale in ((None, 1.0), (_mask(rng, B, T, "holes"), 7.3)):
        act = active_positions(tok, mask, V)
        want = np.where(act[..., None], exact[np.where(act, tok, 0)] * np.float32(scale), np.float32(0))
        out = dp.embedding_lookup(torch.from_numpy(tok).cuda(), to_dev(stored, ti, torch),
                                  mask=None if mask is None else torch.from_numpy(mask).cuda(),
                                  scale=scale, out_dtype=torch.bfloat16 if to == "bf16" else torch.float32)
        if to == "bf16":
            assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.uint16),
                                  f32_to_bf16_bits(want))
        else:
            assert np.array_equal(out.cpu().numpy(), want)


def test_lookup_of_strided_table_rows():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    table = torch.randn(50, 75, device="cuda")
    ids = torch.randint(0, 50, (3, 20), device="cuda", dtype=torch.int32)
    for D in (72, 64, 75, 1):
        out = dp.embedding_lookup(ids, table[:, :D])
        assert torch.equal(out, table[:, :D][ids.long()])


def test_offsets_past_two_and_four_gib():
    """Samples that start more than 2^32 bytes apart, and a table longer than that."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    gap = (1 << 31) + 16                                   # elements between samples
    store = torch.zeros(2 * gap + 4096, dtype=torch.bfloat16, device="cuda")
    G = store.as_strided((3, 4, 64), (gap, 64, 1))
    small = torch.randn(3, 4, 64, device="cuda").bfloat16()
    G.copy_(small)
    ids = torch.tensor([[0, 1, 1, 2], [2, 3, 0, 0], [4, 4, 4, 1]], device="cuda")
    a, an = dp.embedding_clip_accumulate(ids, G, 5, C=3.0, sigma=0.0)
    b, bn = dp.embedding_clip_accumulate(ids, small, 5, C=3.0, sigma=0.0)
    assert torch.equal(a, b) and torch.equal(an, bn)
    rows = (1 << 31) // 1024 + 3                           # 2^31 elements and more
    table = store[: rows * 1024].view(rows, 1024)
    table[-1] = 2.0
    look = torch.tensor([[rows - 1, 0]], device="cuda")
    out = dp.embedding_lookup(look, table)
    assert (out[0, 0] == 2).all() and torch.equal(out[0, 1], table[0])


def test_binding_refuses_bad_arguments():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    ids = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    G = torch.zeros(2, 3, 8, device="cuda")
    table = torch.zeros(5, 8, device="cuda")
    for bad in (lambda: dp.embedding_lookup(ids.float(), table),
                lambda: dp.embedding_lookup(ids[0], table),
                lambda: dp.embedding_lookup(ids.cpu(), table),
                lambda: dp.embedding_lookup(ids, table.t()),
                lambda: dp.embedding_lookup(ids, table.half()),
                lambda: dp.embedding_lookup(ids, table, mask=torch.ones(3, 2, device="cuda")),
                lambda: dp.embedding_lookup(ids, table, out=torch.empty(2, 3, 7, device="cuda")),
                lambda: dp.embedding_lookup(ids, table, scale=float("nan")),
                lambda: dp.embedding_clip_accumulate(ids, G[:1], 5),
                lambda: dp.embedding_clip_accumulate(ids, G, 0),
                lambda: dp.embedding_clip_accumulate(ids, G, 5, C=0.0),
                lambda: dp.embedding_clip_accumulate(ids, G, 5, denom=-1.0),
                lambda: dp.embedding_clip_accumulate(ids, G, 5, accumulate=True),
                lambda: dp.embedding_clip_accumulate(ids, G, 5, grad_out=torch.empty(5, 9, device="cuda")),
                lambda: dp.embedding_clip_accumulate(ids.t(), G.transpose(0, 1), 5),
                lambda: dp.embedding_sqnorms(ids, G, 5, accumulate=True),
                lambda: dp.embedding_scaled_accumulate(ids, G, torch.ones(3, device="cuda"), 5)):
        with pytest.raises((ValueError, TypeError, dp.DpfError)):
            bad()
