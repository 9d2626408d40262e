"""Norms and rotation of queries and keys, their gradients, and dropout, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import attention as oracle
from oracle.dp_linear import widen
from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu
HALF = oracle.HALF


def _np(rng, shape, dtype, f=1.0):
    x = (rng.standard_normal(shape) * f).astype(np.float32)
    return f32_to_bf16_bits(x) if dtype == "bf16" else x


def _dev(torch, x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _close(got, want, bar, half, what):
    err = np.abs(got.double().cpu().numpy() - want)
    bar = bar + half * (np.abs(want) + bar)
    fine = bool(np.isfinite(err).all() and (err <= bar).all())
    assert fine, (what, float(err.max()), float((err / (bar + 1e-300)).max()))


def _rotary(rng, B, T, Hq, Hk, D, pairs, dtype, norm=True, interleaved=False, positions=None, masked=False,
            amplitude=1.0, eps=1e-6, layout=lambda t: t, i32=False):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    q, k, gq, gk = (_np(rng, (B, T, H, D), dtype, f) for H, f in ((Hq, 2.0), (Hk, 0.5), (Hq, 0.1), (Hk, 0.1)))
    wq, wk = ((1 + 0.3 * rng.standard_normal((2, D))).astype(np.float32) if norm else (None, None))
    freqs = 10000.0 ** (-np.arange(pairs) / max(pairs, 1))
    mask = (rng.random((B, T)) < 0.6).astype(np.uint8) if masked else None
    tensors = [layout(to_dev(x, dtype, torch)) for x in (q, k, gq, gk)]
    kw = dict(freqs=_dev(torch, freqs) if pairs else None, mask=_dev(torch, mask), interleaved=interleaved,
              amplitude=amplitude, eps=eps,
              positions=None if positions is None else _dev(torch, positions.astype(np.int32 if i32 else np.int64)))
    weights = (_dev(torch, wq), _dev(torch, wk))
    y = dp.qk_norm_rotary(*tensors[:2], *weights, **kw)
    g = dp.qk_norm_rotary_backward(*tensors[2:], *tensors[:2], *weights, **kw)
    torch.cuda.synchronize()
    for i, (x, w, d) in enumerate(((q, wq, gq), (k, wk, gk))):
        w64 = None if w is None else w.astype(np.float64)
        args = (widen(x, dtype), w64, eps, freqs, positions, amplitude, interleaved, mask)
        _close(y[i], *oracle.oracle_rotary(*args), HALF[dtype], f"output {i}")
        dx, bar, gw, t_gw = oracle.oracle_rotary(*args, dy=widen(d, dtype))
        _close(g[i], dx, bar, HALF[dtype], f"gradient {i}")
        if norm:
            assert g[2 + i].shape == (B, 1, D)
            _close(g[2 + i][:, 0], gw, t_gw, oracle.U, f"weight {i}")
        else:
            assert g[2 + i] is None
    return tensors, weights, kw, y, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [   # B, T, Hq, Hk, D, pairs
    (1, 1, 1, 1, 2, 1), (2, 3, 4, 2, 64, 32), (1, 5, 3, 1, 128, 64), (3, 7, 2, 2, 33, 11), (2, 9, 5, 1, 40, 20),
    (1, 4, 2, 1, 80, 16), (2, 33, 12, 12, 64, 16), (1, 17, 40, 8, 128, 32), (4, 3, 1, 3, 256, 128), (1, 6, 2, 2, 96, 48),
    (2, 5, 7, 3, 45, 22), (1, 3, 2, 2, 255, 100), (1, 2, 3, 3, 24, 8), (5, 1, 2, 1, 1, 0), (2, 40, 3, 2, 72, 0),
])
def test_rotary_matches_oracle(shape, interleaved, norm, dtype):
    if shape[-1] == 0 and not norm:
        pytest.skip("neither norm nor rotation: refused")
    rng = np.random.default_rng(sum(shape))
    _rotary(rng, *shape, dtype, norm=norm, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("far", [100, 70000, 10 ** 6, 2 ** 31 - 1])
def test_far_and_negative_positions(far, dtype):
    rng = np.random.default_rng(far % 97)
    pos = rng.integers(-far, far + 1, (3, 21))
    pos[0, 0], pos[1, 1], pos[2, 2] = far, -far, 0
    _rotary(rng, 3, 21, 4, 2, 64, 32, dtype, positions=pos, i32=far < 2 ** 31)
    _rotary(rng, 3, 21, 3, 1, 30, 10, dtype, positions=pos, interleaved=True, masked=True, amplitude=1.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotary_masks_strides_and_many_rows(dtype):
    rng = np.random.default_rng(5)
    for layout in (lambda t: t.transpose(1, 2).contiguous().transpose(1, 2),
                   lambda t: t.new_full((t.shape[0], t.shape[1], t.shape[2] + 1, t.shape[3] + 4), 9.0)
                   [:, :, 1:, 4:].copy_(t),
                   lambda t: t.new_full((t.shape[0], t.shape[1], t.shape[2], t.shape[3] + 1), 9.0)[..., 1:].copy_(t)):
        _rotary(rng, 2, 19, 6, 2, 64, 32, dtype, masked=True, layout=layout)
    _rotary(rng, 2, 1300, 5, 2, 64, 32, dtype, masked=True)
    _rotary(rng, 1, 2500, 3, 1, 48, 24, dtype, interleaved=True)


def test_rotary_masked_rows_are_not_read():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(6)
    for D in (64, 33):
        (q, k, gq, gk), w, kw, y, g = _rotary(rng, 2, 30, 3, 2, D, D // 2, "bf16", masked=True)
        off = kw["mask"] == 0
        for x in (q, k, gq, gk):
            x[off] = float("nan")
        y2 = dp.qk_norm_rotary(q, k, *w, **kw)
        g2 = dp.qk_norm_rotary_backward(gq, gk, q, k, *w, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*y, *g), (*y2, *g2)))
        assert not y[0][off].any() and not g[1][off].any()


@pytest.mark.parametrize("D", [64, 33])
def test_rotary_in_place_and_on_parts_of_one_array(D):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(7)
    B, T, Hq, Hk = 2, 50, 4, 2
    rows = to_dev(_np(rng, (B, T, Hq + 2 * Hk, D), "bf16"), "bf16", torch)
    q, k, v = rows.split([Hq, Hk, Hk], dim=2)
    d = to_dev(_np(rng, (B, T, Hq + Hk, D), "bf16"), "bf16", torch)
    w = _dev(torch, (1 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    freqs, amplitude = dp.rotary_frequencies(2 * (D // 4), scaling="yarn", factor=4.0, length=64)
    kw = dict(freqs=freqs, amplitude=amplitude)
    want = dp.qk_norm_rotary(q, k, w, w, **kw)
    grads = dp.qk_norm_rotary_backward(d[:, :, :Hq], d[:, :, Hq:], q, k, w, w, **kw)
    values = v.clone()
    d2 = d.clone()
    got = dp.qk_norm_rotary_backward(d2[:, :, :Hq], d2[:, :, Hq:], q, k, w, w, **kw, dq=d2[:, :, :Hq],
                                     dk=d2[:, :, Hq:])
    dp.qk_norm_rotary(q, k, w, w, **kw, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, values)
    assert all(torch.equal(a, b) for a, b in zip(grads, got))


def test_weight_gradients_clip_as_a_linear_of_one_input():
    """The per-sample gradients through the library's own clipping calls."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(8)
    _, _, _, _, g = _rotary(rng, 6, 20, 4, 2, 64, 32, "f32", masked=True)
    per = g.dq_weight
    ones = torch.ones((6, 1, 1), device="cuda")
    norms = per[:, 0].double().norm(dim=1)
    C = float(norms.median())
    out, n = dp.linear_clip_accumulate(ones, per, C=C, sigma=0.0)
    want = (per[:, 0].double() * (C / norms).clamp(max=1.0)[:, None]).sum(0) / 6
    # sums of 64 squares, of 6 terms, and their products: 80 roundings at most
    assert ((n.double() - norms).abs() <= 80 * 2.0 ** -24 * norms).all()
    assert ((out[:, 0].double() - want).abs() <= 80 * 2.0 ** -24 * per[:, 0].double().abs().sum(0) / 6).all()


def test_rotary_repeats_replays_and_other_streams():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(9)
    (q, k, gq, gk), w, kw, y, g = _rotary(rng, 2, 300, 4, 2, 64, 32, "bf16", masked=True)

    def run():
        return [*dp.qk_norm_rotary(q, k, *w, **kw), *dp.qk_norm_rotary_backward(gq, gk, q, k, *w, **kw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*y, *g), side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for rep in range(4):
        for t, H in ((q, 4), (k, 2), (gq, 4), (gk, 2)):
            t.copy_(to_dev(_np(rng, (2, 300, H, 64), "bf16"), "bf16", torch))
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), rep


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999, 2.0 ** -16])
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 8), (1, 5, 7), (3, 4, 64), (2, 9, 100), (1, 1, 1000), (4, 33, 24)])
def test_dropout_matches_oracle(shape, p, dtype):
    """What is kept exactly; the values to one rounding of the product, one of the sum and one to
    the type."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape))
    x, r = _np(rng, shape, dtype), _np(rng, shape, dtype, 3.0)
    seed, offset = int(rng.integers(0, 2 ** 63)), int(rng.integers(0, 2 ** 40))
    mask = (rng.random(shape[:2]) < 0.7).astype(np.uint8)
    tx, tr = to_dev(x, dtype, torch), to_dev(r, dtype, torch)
    for residual, m in ((None, None), (tr, None), (None, mask), (tr, mask)):
        y = dp.dropout(tx, p, seed, offset, residual=residual, mask=_dev(torch, m))
        torch.cuda.synchronize()
        want, kept = oracle.oracle_dropout(widen(x, dtype), p, seed, offset,
                                           None if residual is None else widen(r, dtype), m)
        got = y.double().cpu().numpy()
        factor = 65536.0 / (65536 - round(65536 * p))
        bar = 3 * oracle.U * (np.abs(widen(x, dtype)) * factor + np.abs(want))
        assert (np.abs(got - want) <= bar + HALF[dtype] * (np.abs(want) + bar)).all()
        if residual is None:
            live = np.ones(shape[:2], bool) if m is None else m != 0
            assert not got[~(kept & live[..., None])].any()


def test_dropout_rates_and_streams_apart():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    x = torch.ones((4, 256, 1024), device="cuda")
    n = x.numel()
    for p in (0.05, 0.3, 0.5):
        kept = (dp.dropout(x, p, seed=11, offset=5) != 0).double()
        # the mean of n draws of variance p (1 - p): six standard deviations
        assert abs(float(kept.mean()) - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -17
    a = dp.dropout(x, 0.5, seed=11, offset=0)
    b = dp.dropout(x, 0.5, seed=11, offset=dp.dropout_blocks(n))
    both = ((a != 0) & (b != 0)).double().mean()
    assert abs(float(both) - 0.25) < 6 * (3.0 / 16 / n) ** 0.5
    # a later offset draws the later entries' bits
    c = dp.dropout(x, 0.5, seed=11, offset=1024 // 8)
    assert torch.equal(c.reshape(-1)[: n - 1024], a.reshape(-1)[1024:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_strides_places_and_gradient(dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(3)
    for D in (40, 41):
        x = to_dev(_np(rng, (3, 11, D), dtype), dtype, torch)
        r = to_dev(_np(rng, (3, 11, D), dtype), dtype, torch)
        want = dp.dropout(x, 0.3, 5, 9, residual=r)
        wide = x.new_full((3, 13, D + 5), float("nan"))
        part = wide[:, 1:-1, 3: D + 3]
        part.copy_(x)
        assert torch.equal(dp.dropout(part, 0.3, 5, 9, residual=r), want)
        dp.dropout(part, 0.3, 5, 9, residual=r, out=part)
        torch.cuda.synchronize()
        assert torch.equal(part, want) and int(wide.isnan().sum()) == wide.numel() - part.numel()
        r2 = r.clone()
        assert torch.equal(dp.dropout(x, 0.3, 5, 9, residual=r2, out=r2), want)
        # the gradient: the same entries, the same factor
        dy = to_dev(_np(rng, (3, 11, D), dtype), dtype, torch)
        dx = dp.dropout(dy, 0.3, 5, 9)
        keep = dp.dropout(torch.ones_like(x, dtype=torch.float32), 0.3, 5, 9)
        assert torch.equal(dx, (dy.float() * keep).to(dx.dtype))
        # by differences: dropout is linear in x
        base = dp.dropout(x.float(), 0.3, 5, 9)
        moved = dp.dropout(x.float() + 0.5, 0.3, 5, 9)
        assert ((moved - base) - 0.5 * keep).abs().max() <= 4 * 2.0 ** -24 * float(moved.abs().max() + 1)


def test_dropout_masked_rows_are_not_read_and_replays():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(4)
    for D in (64, 33):
        x = to_dev(_np(rng, (2, 9, D), "bf16"), "bf16", torch)
        r = x.clone()
        mask = _dev(torch, (rng.random((2, 9)) < 0.5).astype(np.uint8))
        want = dp.dropout(x, 0.2, 1, 2, residual=r, mask=mask)
        x[mask == 0] = float("nan")
        r[mask == 0] = float("inf")
        got = dp.dropout(x, 0.2, 1, 2, residual=r, mask=mask)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and not got[mask == 0].any()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = dp.dropout(x, 0.2, 1, 2, residual=r, mask=mask)
        for _ in range(3):
            x.copy_(to_dev(_np(rng, (2, 9, D), "bf16"), "bf16", torch))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, dp.dropout(x, 0.2, 1, 2, residual=r, mask=mask))


def test_dropout_of_many_entries():
    """More entries than 2^32: each block of entries still has its own bits."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    D = 4096
    T = (1 << 20) + 3
    x = torch.ones((1, T, D), dtype=torch.bfloat16, device="cuda")
    y = dp.dropout(x, 0.5, seed=9, offset=1 << 33, out=x)
    tail = dp.dropout(torch.ones((1, 3, D), dtype=torch.bfloat16, device="cuda"), 0.5, seed=9,
                      offset=(1 << 33) + (1 << 20) * D // 8)
    torch.cuda.synchronize()
    assert torch.equal(y[:, 1 << 20:], tail)
