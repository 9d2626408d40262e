"""Attention and its gradients against the fp64 oracle, whose bars follow the computation's
roundings (oracle/attention.py)."""
import numpy as np
import pytest

from oracle import attention as oracle
from oracle.dp_linear import widen
from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _draw(rng, B, Tq, Tk, Hq, Hkv, D, dtype, spread=1.5):
    """q, k, v, dout as numpy in the type's storage."""
    arrays = [rng.standard_normal((B, T, H, D)).astype(np.float32) * f
              for T, H, f in ((Tq, Hq, spread), (Tk, Hkv, spread), (Tk, Hkv, 1.0), (Tq, Hq, 0.1))]
    return [f32_to_bf16_bits(x) if dtype == "bf16" else x for x in arrays]


def _mask(rng, kind, B, T):
    if kind is None:
        return None
    if kind == "prefix":
        n = rng.integers(0, T + 1, B)
        n[0] = T
        return (np.arange(T)[None] < n[:, None]).astype(np.uint8)
    if kind == "left":
        n = rng.integers(1, T + 1, B)
        return (np.arange(T)[None] >= T - n[:, None]).astype(np.uint8)
    return (rng.random((B, T)) < 0.6).astype(np.uint8)


def _segments(rng, B, T, n):
    """Document numbers with gaps, some documents of one position."""
    cuts = np.sort(rng.integers(0, T, (B, n)), 1)
    return ((np.arange(T)[None, :, None] >= cuts[:, None, :]).sum(-1) * 3 - 5).astype(np.int32)


def _dev(torch, x):
    return None if x is None else torch.from_numpy(x).cuda()


def _value(t):
    return t.double().cpu().numpy()


def _close(got, want, bar, what):
    err = np.abs(_value(got) - want)
    finite = bool(np.isfinite(err).all())
    assert finite, what
    over = err > bar
    some = bool(over.any())
    assert not some, (what, float(err[over].max()), float(bar[over].min()), int(over.sum()))


def _check(q, k, v, dout, dtype, mask=None, segments=None, causal=True, scale=None, back=True, layout=None):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    place = layout or (lambda t, name: t)
    tq, tk, tv, td = (place(to_dev(x, dtype, torch), n) for x, n in zip((q, k, v, dout), "qkvd"))
    m, s = _dev(torch, mask), _dev(torch, segments)
    r = dp.attention(tq, tk, tv, mask=m, segments=s, causal=causal, scale=scale)
    grads = dp.attention_backward(td, tq, tk, tv, r.out, r.lse, mask=m, segments=s, causal=causal,
                                  scale=scale) if back else ()
    torch.cuda.synchronize()
    f = q.shape[3] ** -0.5 if scale is None else scale
    wide = [widen(x, dtype) for x in (q, k, v, dout)]
    want = oracle.oracle_attention(*wide[:3], mask, segments, causal, f, dtype, dout=wide[3] if back else None)
    for name, got, (value, bar) in zip(("out", "lse", "dq", "dk", "dv"), (*r, *grads), want):
        _close(got, value, bar, name)
    return r, grads


SHAPES = [  # B, Tq, Tk, Hq, Hkv, D
    (1, 1, 1, 1, 1, 1), (2, 2, 2, 2, 1, 8), (1, 31, 31, 1, 1, 64), (2, 32, 32, 3, 1, 33),
    (1, 33, 33, 4, 2, 40), (2, 63, 63, 2, 2, 128), (1, 64, 64, 5, 1, 45), (1, 65, 65, 2, 1, 72),
    (3, 127, 127, 2, 2, 64), (1, 128, 128, 4, 1, 128), (2, 129, 129, 1, 1, 100), (1, 200, 200, 3, 3, 96),
    (1, 257, 257, 8, 2, 64), (2, 300, 300, 2, 1, 127), (9, 5, 5, 6, 3, 16), (1, 513, 513, 1, 1, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_oracle(shape, causal, dtype):
    rng = np.random.default_rng(sum(shape))
    _check(*_draw(rng, *shape, dtype), dtype, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("docs", [0, 1, 4, 40])
@pytest.mark.parametrize("kind", [None, "prefix", "left", "holes"])
def test_masks_and_segments(kind, docs, causal, dtype):
    rng = np.random.default_rng(docs + 7)
    for B, T, Hq, Hkv, D in ((3, 70, 2, 1, 64), (2, 200, 2, 2, 40), (4, 5, 3, 1, 24), (1, 331, 1, 1, 128)):
        _check(*_draw(rng, B, T, T, Hq, Hkv, D, dtype), dtype, mask=_mask(rng, kind, B, T),
               segments=_segments(rng, B, T, docs) if docs else None, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [
    (2, 1, 1, 4, 2, 64), (2, 1, 31, 8, 1, 64), (1, 1, 257, 5, 5, 128), (3, 1, 1000, 8, 2, 40), (1, 3, 700, 6, 2, 45),
    (1, 8, 129, 4, 1, 128), (1, 32, 400, 1, 1, 96), (1, 33, 400, 1, 1, 96), (2, 11, 90, 3, 1, 64), (1, 1, 5000, 32, 1, 128),
    (1, 100, 131, 2, 1, 64), (1, 200, 201, 1, 1, 128), (1, 130, 700, 2, 2, 33),
])
def test_queries_at_the_end_of_the_keys(shape, dtype):
    """New positions over those before them: the keys split over workgroups, or not."""
    rng = np.random.default_rng(sum(shape))
    B, Tq, Tk = shape[:3]
    arrays = _draw(rng, *shape, dtype)
    _check(*arrays, dtype)
    _check(*arrays, dtype, mask=_mask(rng, "left", B, Tk), causal=False)
    if Tk > 4:
        _check(*arrays, dtype, mask=_mask(rng, "holes", B, Tk), segments=_segments(rng, B, Tk, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_and_large_scores(dtype):
    """Scores that leave most weights at zero, that rise along the keys (the maximum keeps being
    replaced) and that are all equal."""
    rng = np.random.default_rng(2)
    q, k, v, d = _draw(rng, 2, 150, 150, 2, 1, 64, "f32")
    rise = k * np.linspace(0.01, 3.0, 150, dtype=np.float32)[None, :, None, None]
    same = np.broadcast_to(k[:, :1], k.shape).copy()
    for keys, scale in ((k, 3.0), (k, 1e-3), (rise, 1.0), (rise[:, ::-1].copy(), 1.0), (same, None)):
        arrays = [f32_to_bf16_bits(x) if dtype == "bf16" else x for x in (q, keys, v, d)]
        _check(*arrays, dtype, causal=False, scale=scale)


def _bhtd(t, name):
    """The same values, stored [B, H, T, D]."""
    return t.transpose(1, 2).contiguous().transpose(1, 2)


def _spread(t, name):
    """The same values between others, rows at odd offsets."""
    B, T, H, D = t.shape
    big = t.new_full((B, T + 1, H + 2, D + 3), float("nan"))
    part = big[:, 1:, 1: H + 1, 1: D + 1]
    part.copy_(t)
    return part


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [_bhtd, _spread])
@pytest.mark.parametrize("D", [64, 45, 128])
def test_layouts(D, layout, dtype):
    rng = np.random.default_rng(D)
    _check(*_draw(rng, 2, 140, 140, 4, 2, D, dtype), dtype, mask=_mask(rng, "prefix", 2, 140), layout=layout)
    _check(*_draw(rng, 2, 3, 90, 4, 2, D, dtype), dtype, layout=layout)


def test_broadcast_inputs():
    """One head of keys seen as several (stride 0), one sample's keys as the batch's."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(0)
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, 3, 70, 70, 4, 1, 64, "bf16"))
    a = dp.attention(q, k[:1].expand(3, 70, 4, 64), v[:1].expand(3, 70, 4, 64))
    b = dp.attention(q, k[:1].repeat(3, 1, 4, 1), v[:1].repeat(3, 1, 4, 1))
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("D", [64, 45])
def test_gradients_into_parts_of_one_array(D):
    """dq, dk and dv as parts of a fused projection's gradient, and out within a larger array:
    the same values, and nothing written around them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(D)
    B, T, Hq, Hkv = 2, 131, 4, 2
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, B, T, T, Hq, Hkv, D, "bf16"))
    mask = _dev(torch, _mask(rng, "prefix", B, T))
    plain = dp.attention(q, k, v, mask=mask)
    grads = dp.attention_backward(d, q, k, v, plain.out, plain.lse, mask=mask)
    fused = torch.full((B, T + 2, Hq + 2 * Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    parts = [p[:, 1:-1] for p in fused.split([Hq, Hkv, Hkv], dim=2)]
    dp.attention_backward(d, q, k, v, plain.out, plain.lse, mask=mask, dq=parts[0], dk=parts[1], dv=parts[2])
    rows = torch.full((B, T, Hq + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    r = dp.attention(q, k, v, mask=mask, out=rows[:, :, 1:-1])
    torch.cuda.synchronize()
    for a, b in zip(parts, grads):
        assert torch.equal(a, b)
    assert torch.equal(r.out, plain.out) and torch.equal(r.lse, plain.lse)
    assert (fused[:, 0] == 7.0).all() and (fused[:, -1] == 7.0).all()
    assert (rows[:, :, 0] == 7.0).all() and (rows[:, :, -1] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 150, 150, 2, 1, 64), (2, 2, 150, 2, 1, 128), (2, 37, 37, 2, 2, 45)])
def test_what_masked_places_hold_does_not_matter(shape, dtype):
    """NaN, infinities and the type's extremes in masked rows of every tensor: bitwise the result
    with zeros there, and zeros where the rows are masked."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(1)
    B, Tq, Tk = shape[:3]
    q, k, v, d = (to_dev(x, dtype, torch) for x in _draw(rng, *shape, dtype))
    for kind in ("prefix", "holes", "left"):
        m = _mask(rng, kind, B, Tk)
        m[1, : Tk // 2] = 0
        mask = _dev(torch, m)
        off = mask == 0
        results = []
        for fill in (0.0, float("nan"), float("inf"), torch.finfo(q.dtype).min):
            Q, K, V, G = (x.clone() for x in (q, k, v, d))
            for x, dead in ((Q, off[:, Tk - Tq:]), (K, off), (V, off), (G, off[:, Tk - Tq:])):
                x[dead] = fill
            r = dp.attention(Q, K, V, mask=mask)
            out = r.out.clone()
            out[off[:, Tk - Tq:]] = fill
            lse = r.lse.clone()
            lse.transpose(1, 2)[off[:, Tk - Tq:]] = fill
            results.append([*r, *dp.attention_backward(G, Q, K, V, out, lse, mask=mask)])
        torch.cuda.synchronize()
        for other in results[1:]:
            for a, b in zip(results[0], other):
                assert torch.equal(a, b)
        for x, dead in zip(results[0], (off[:, Tk - Tq:], None, off[:, Tk - Tq:], off, off)):
            if dead is not None:
                assert not x[dead].any()
        assert not results[0][1].transpose(1, 2)[off[:, Tk - Tq:]].any()


def test_empty_samples():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for T, Tk in ((200, 200), (1, 200), (1, 1)):
        q = torch.full((2, T, 2, 64), float("nan"), device="cuda")
        k = torch.full((2, Tk, 1, 64), float("nan"), device="cuda")
        mask = torch.zeros((2, Tk), dtype=torch.uint8, device="cuda")
        r = dp.attention(q, k, k, mask=mask)
        g = dp.attention_backward(q, q, k, k, r.out, r.lse, mask=mask)
        torch.cuda.synchronize()
        assert not any(x.any() for x in (*r, *g))


def test_a_sample_keeps_its_nan():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(4)
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, 3, 100, 100, 2, 2, 64, "bf16"))
    clean = dp.attention(q, k, v)
    want = dp.attention_backward(d, q, k, v, clean.out, clean.lse)
    v2, k2 = v.clone(), k.clone()
    v2[1, 5], k2[1, 9] = float("nan"), float("inf")
    r = dp.attention(q, k2, v2)
    got = dp.attention_backward(d, q, k2, v2, r.out, r.lse)
    torch.cuda.synchronize()
    for a, b in zip((clean.out, clean.lse, *want), (r.out, r.lse, *got)):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert r.out[1, 5:].isnan().all() and r.out[1, 99].isnan().all()


@pytest.mark.parametrize("T", [1, 7, 300])
def test_one_key_gives_its_value_and_no_gradient(T):
    """Segments of one position: out = v exactly, dq = dk = 0, dv = dout summed over the group."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(T)
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, 2, T, T, 4, 2, 64, "bf16"))
    seg = torch.arange(T, dtype=torch.int32, device="cuda").expand(2, T).contiguous()
    for causal in (True, False):
        r = dp.attention(q, k, v, segments=seg, causal=causal)
        dq, dk, dv = dp.attention_backward(d, q, k, v, r.out, r.lse, segments=seg, causal=causal)
        torch.cuda.synchronize()
        assert torch.equal(r.out, v.repeat_interleave(2, 2)) and not dq.any() and not dk.any()
        want = d.double().reshape(2, T, 2, 2, 64).sum(3)
        assert ((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all()


def test_repeats_bitwise():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(6)
    for shape in ((2, 300, 300, 4, 2, 128), (1, 2, 3000, 8, 1, 64)):
        q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, *shape, "bf16"))
        first = None
        for _ in range(5):
            r = dp.attention(q, k, v)
            g = dp.attention_backward(d, q, k, v, r.out, r.lse)
            torch.cuda.synchronize()
            if first is None:
                first = (*r, *g)
            for a, b in zip(first, (*r, *g)):
                assert torch.equal(a, b)


def test_decreasing_segments_stay_within_the_tensors():
    """Out of contract, yet only finite values of the same sample come out."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(8)
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, 2, 333, 333, 2, 1, 64, "bf16"))
    seg = _dev(torch, rng.integers(-2 ** 31, 2 ** 31 - 1, (2, 333)).astype(np.int32))
    r = dp.attention(q, k, v, segments=seg)
    g = dp.attention_backward(d, q, k, v, r.out, r.lse, segments=seg)
    torch.cuda.synchronize()
    assert all(x.isfinite().all() for x in (*r, *g))


def test_extreme_segment_numbers():
    rng = np.random.default_rng(9)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    seg = np.array([[lo] * 40 + [0] * 50 + [hi] * 60, [hi] * 150], np.int32)
    for causal in (True, False):
        _check(*_draw(rng, 2, 150, 150, 1, 1, 64, "bf16"), "bf16", segments=seg, causal=causal)


def test_offsets_past_32_bits():
    """Samples and heads whose entries lie more than 2^32 elements apart."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(10)
    B, T, H, D = 2, 70, 2, 64
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, B, T, T, H, H, D, "bf16"))
    far = (1 << 32) + 64
    pool = torch.empty(far + (1 << 31) + 4 * T * D, dtype=torch.bfloat16, device="cuda")
    strides = (far, D, (1 << 31) + 64, 1)

    def put(x):
        y = pool.as_strided(x.shape, strides)
        y.copy_(x)
        return y
    want = dp.attention(q, k, v)
    grads = dp.attention_backward(d, q, k, v, want.out, want.lse)
    for i, x in enumerate((q, k, v)):
        args = [q, k, v]
        args[i] = put(x)
        r = dp.attention(*args)
        g = dp.attention_backward(d, *args, r.out, r.lse)
        torch.cuda.synchronize()
        assert torch.equal(r.out, want.out) and all(torch.equal(a, b) for a, b in zip(g, grads))
    out = pool.as_strided(q.shape, strides)
    out.zero_()
    r = dp.attention(q, k, v, out=out)
    torch.cuda.synchronize()
    assert torch.equal(r.out, want.out)


def test_on_another_stream_and_two_at_once():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(11)
    shape = (2, 400, 400, 4, 2, 64)
    q, k, v, d = (to_dev(x, "bf16", torch) for x in _draw(rng, *shape, "bf16"))
    masks = [_dev(torch, _mask(rng, kind, 2, 400)) for kind in ("prefix", "holes")]
    want = []
    for m in masks:
        r = dp.attention(q, k, v, mask=m)
        want.append((*r, *dp.attention_backward(d, q, k, v, r.out, r.lse, mask=m)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in masks]
    got = [[], []]
    for _ in range(4):
        for i, (s, m) in enumerate(zip(streams, masks)):
            r = dp.attention(q, k, v, mask=m, stream=s)
            with torch.cuda.stream(s):
                got[i].append((*r, *dp.attention_backward(d, q, k, v, r.out, r.lse, mask=m)))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, run))


@pytest.mark.parametrize("D", [64, 45])
def test_captured_and_replayed(D):
    """Two graphs, each with a forward and a backward pass, replayed in turn between eager calls:
    every replay gives the eager result for what the inputs then hold."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(12)
    cases = []
    for shape, kind in (((2, 200, 200, 4, 2, D), "prefix"), ((3, 1, 900, 8, 2, D), "left")):
        B, Tq, Tk = shape[:3]
        tensors = [to_dev(x, "bf16", torch) for x in _draw(rng, *shape, "bf16")]
        mask = _dev(torch, _mask(rng, kind, B, Tk))
        seg = torch.zeros((B, Tk), dtype=torch.int32, device="cuda")

        def run(t=tensors, m=mask, s=seg):
            r = dp.attention(*t[:3], mask=m, segments=s)
            return [*r, *dp.attention_backward(t[3], *t[:3], r.out, r.lse, mask=m, segments=s)]
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        cases.append((shape, tensors, run, graph, out))
    for rep in range(4):
        for shape, tensors, run, graph, out in cases:
            for t, x in zip(tensors, _draw(rng, *shape, "bf16")):
                t.copy_(to_dev(x, "bf16", torch))
            graph.replay()
            torch.cuda.synchronize()
            eager = run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager)), (rep, shape)


def test_workspace_limit_fails_before_anything_is_written():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    q = torch.randn((1, 300, 2, 64), device="cuda")
    mask = torch.ones((1, 300), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 5.0)
    dp.set_option("workspace_limit_bytes", 16)
    try:
        with pytest.raises(dp.DpfError) as e:
            dp.attention(q, q, q, mask=mask, out=out)
    finally:
        dp.set_option("workspace_limit_bytes", 0)
    assert e.value.status == 3
    torch.cuda.synchronize()
    assert (out == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longer_sequences(dtype):
    """Many tiles of keys, three documents and a ragged batch, against the oracle."""
    rng = np.random.default_rng(13)
    _check(*_draw(rng, 1, 1500, 1500, 2, 1, 128, dtype), dtype)
    _check(*_draw(rng, 2, 1111, 1111, 1, 1, 64, dtype), dtype, mask=_mask(rng, "prefix", 2, 1111),
           segments=_segments(rng, 2, 1111, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 45, 128, 99])
def test_many_workgroups(D, dtype):
    """More heads than compute units take at a time, of a length that ends inside a tile: the
    backward pass then gives each wave keys of its own."""
    rng = np.random.default_rng(14)
    _check(*_draw(rng, 5, 70, 70, 54, 27, D, dtype), dtype, mask=_mask(rng, "prefix", 5, 70))
    _check(*_draw(rng, 33, 33, 41, 4, 4, D, dtype), dtype)
    _check(*_draw(rng, 29, 130, 130, 3, 3, D, dtype), dtype, causal=False,
           segments=_segments(rng, 29, 130, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -30])
def test_smallest_scales(scale, dtype):
    """All weights of a row alike: lse = log n, lse / scale up to 10^20.  (The scores' sums then
    round at lse / scale, D = 16 terms of half a step of lse <= 5.1 each: 82 u of a weight, within
    the bar's Tk + 16 = 166.)"""
    rng = np.random.default_rng(15)
    _check(*_draw(rng, 2, 150, 150, 2, 1, 16, dtype), dtype, mask=_mask(rng, "holes", 2, 150), scale=scale)


@pytest.mark.parametrize("D", [64, 45, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_queries_beside_nan(D, dtype):
    """Rows whose own mask byte is 0 give exact zeros and take part in no gradient, though the rows
    beside them, in the same tile, hold NaN; other samples are not touched."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(16)
    B, T, H = 2, 70, 2
    q, k, v, g = (to_dev(x, dtype, torch) for x in _draw(rng, B, T, T, H, H, D, dtype))
    mask = np.ones((B, T), np.uint8)
    mask[:, 1::2] = 0
    m = _dev(torch, mask)
    clean = dp.attention(q, k, v, mask=m)
    clean_grads = dp.attention_backward(g, q, k, v, clean.out, clean.lse, mask=m)
    for t in (q, k, v, g):
        t[0, 0] = float("nan")          # an active position of the first sample
        t[:, 1::2] = float("nan")       # masked ones of both
    r = dp.attention(q, k, v, mask=m)
    grads = dp.attention_backward(g, q, k, v, r.out, r.lse, mask=m)
    torch.cuda.synchronize()
    for x in (r.out, *grads):
        assert (x[:, 1::2] == 0).all()
    assert (r.lse[:, :, 1::2] == 0).all()
    for x, y in zip((r.out, r.lse, *grads), (clean.out, clean.lse, *clean_grads)):
        assert torch.equal(x[1], y[1])


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_far_from_zero(sign, dtype):
    """Every score near -300 or 300, where e^s is 0 or infinite in float32, with masked keys and
    queries in each tile: only differences of scores may be raised."""
    rng = np.random.default_rng(17)
    q, k, v, dout = _draw(rng, 2, 100, 100, 2, 1, 64, "f32", spread=0.1)
    q[..., 0], k[..., 0] = 48.0, sign * 50.0
    if dtype == "bf16":
        q, k, v, dout = (f32_to_bf16_bits(x) for x in (q, k, v, dout))
    _check(q, k, v, dout, dtype, mask=_mask(rng, "holes", 2, 100))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 45, 128])
def test_single_tokens_of_many_sequences(D, dtype):
    """More heads than compute units, so that no head's keys are split."""
    rng = np.random.default_rng(18)
    _check(*_draw(rng, 300, 1, 70, 2, 1, D, dtype), dtype, mask=_mask(rng, "left", 300, 70), back=False)
    _check(*_draw(rng, 260, 2, 33, 1, 1, D, dtype), dtype, back=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens_over_a_long_cache(dtype):
    """Keys split as often as they are at most."""
    rng = np.random.default_rng(19)
    _check(*_draw(rng, 1, 1, 17003, 4, 1, 64, dtype), dtype, back=False)
    _check(*_draw(rng, 1, 3, 17003, 2, 1, 16, dtype), dtype, mask=_mask(rng, "holes", 1, 17003), back=False)


@pytest.mark.parametrize("kind", ["prefix", "left", "holes"])
@pytest.mark.parametrize("T", [63, 64, 65, 128, 191, 192, 255, 256, 257])
def test_masks_of_short_samples(T, kind):
    """Up to 256 positions the forward pass reads the mask itself."""
    rng = np.random.default_rng(20)
    for causal, Tq in ((True, T), (False, T), (True, 33)):
        _check(*_draw(rng, 3, Tq, T, 2, 2, 64, "bf16"), "bf16", mask=_mask(rng, kind, 3, T), causal=causal)
    _check(*_draw(rng, 2, T, T, 2, 1, 24, "f32"), "f32", mask=_mask(rng, kind, 2, T))


@pytest.mark.parametrize("D", [64, 45, 128])
def test_short_samples_of_many_heads(D):
    """float32, up to 32 keys or queries, more workgroups than compute units: the waves share them."""
    rng = np.random.default_rng(21)
    _check(*_draw(rng, 40, 7, 7, 28, 7, D, "f32"), "f32", mask=_mask(rng, "left", 40, 7))
    _check(*_draw(rng, 70, 5, 90, 4, 4, D, "f32"), "f32", causal=False)
