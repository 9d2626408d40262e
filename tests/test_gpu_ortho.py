"""Newton-Schulz orthogonalisation and the optimizer step on it against the fp64 oracle.

Bar: the accuracy of float32 products.  The same iteration in numpy float32 has an error
e32 (Frobenius norm) that the iteration itself amplifies, by up to a^steps where singular
values are small, so no fixed number fits; the kernels may have 4 e32 (their sums run in
another order) plus 8 u ||X||_F for the operands' 22 bits, u = 2^-24.  bf16 results are the
float32 ones rounded, bit for bit.
"""
import numpy as np
import pytest

from oracle import optim
from tests.gpu_helpers import need_gpu
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
COEFFS = (3.4445, -4.7750, 2.0315)


def _bar(M, steps, coeffs, eps):
    ref = optim.newton_schulz(M, steps, coeffs, eps)
    plain = optim.newton_schulz(M, steps, coeffs, eps, np.float32).astype(np.float64)
    return ref, 4 * np.linalg.norm(plain - ref) + 8 * U * np.linalg.norm(ref)


def _matrix(rng, R, C, kind):
    if kind == "lowrank":
        k = max(1, min(R, C) // 4)
        M = rng.standard_normal((R, k)) @ rng.standard_normal((k, C)) + 1e-2 * rng.standard_normal((R, C))
    elif kind == "spike":
        M = rng.standard_normal((R, C))
        M[0] *= 100.0
    else:
        M = rng.standard_normal((R, C))
    return (M * 1e-3).astype(np.float32)


@pytest.mark.parametrize("kind", ["full", "lowrank", "spike"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 50), (50, 1), (3, 5), (64, 32), (32, 64), (63, 65),
                                   (65, 63), (64, 64), (128, 128), (129, 64), (200, 300), (300, 200),
                                   (257, 257), (100, 1001), (1001, 100), (256, 768), (520, 512)])
def test_matches_oracle(shape, kind):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape))
    M = _matrix(rng, *shape, kind)
    for steps in (1, 5):
        out = dp.orthogonalize(torch.from_numpy(M).cuda(), steps=steps).cpu().numpy()
        ref, bar = _bar(M, steps, COEFFS, 1e-7)
        err = np.linalg.norm(out - ref)
        assert err <= bar, (steps, err, bar)


@pytest.mark.parametrize("shape", [(1024, 1024), (700, 2050), (2050, 700)])
def test_larger_matrices(shape):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(1)
    M = _matrix(rng, *shape, "full")
    out = dp.orthogonalize(torch.from_numpy(M).cuda()).cpu().numpy()
    ref, bar = _bar(M, 5, COEFFS, 1e-7)
    assert np.linalg.norm(out - ref) <= bar


@pytest.mark.parametrize("shape", [(40, 24), (96, 100), (300, 140)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_a_stack_is_its_matrices(n, shape):
    """Every matrix of a stack against the oracle, each with its own norm."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(n)
    M = np.stack([_matrix(rng, *shape, "full") * 10.0 ** (k % 5) for k in range(n)])
    out = dp.orthogonalize(torch.from_numpy(M).cuda()).cpu().numpy()
    for k in range(n):
        ref, bar = _bar(M[k], 5, COEFFS, 1e-7)
        assert np.linalg.norm(out[k] - ref) <= bar


@pytest.mark.parametrize("shape", [(33, 70), (128, 64), (2, 50, 31)])
def test_bf16_is_the_float32_result_rounded(shape):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(5)
    M = f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    t = torch.from_numpy(M.view(np.int16)).view(torch.bfloat16).cuda()
    a = dp.orthogonalize(t).view(torch.int16).cpu().numpy().view(np.uint16)
    b = dp.orthogonalize(torch.from_numpy(bf16_bits_to_f32(M)).cuda()).cpu().numpy()
    assert np.array_equal(a, f32_to_bf16_bits(b))


def test_converges_to_the_polar_factor():
    """With (1.5, -0.5, 0) and enough steps the limit is U V^T of the singular value decomposition."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(2)
    for shape in ((80, 120), (120, 80), (64, 64)):
        q1, _ = np.linalg.qr(rng.standard_normal((shape[0], min(shape))))
        q2, _ = np.linalg.qr(rng.standard_normal((shape[1], min(shape))))
        M = (q1 * np.linspace(0.3, 1.0, min(shape))) @ q2.T
        out = dp.orthogonalize(torch.from_numpy(M.astype(np.float32)).cuda(), steps=24,
                               coeffs=(1.5, -0.5, 0.0)).cpu().numpy()
        ref, bar = _bar(M.astype(np.float32), 24, (1.5, -0.5, 0.0), 1e-7)
        assert np.linalg.norm(out - ref) <= bar
        # the iteration's own limit: singular values of 1 to within float32 of each entry
        assert np.linalg.norm(out - q1 @ q2.T) <= bar + 1e-6 * np.sqrt(min(shape))


def test_zero_tiny_huge_and_not_finite():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(3)
    M = rng.standard_normal((6, 40, 70)).astype(np.float32)
    M[0] = 0.0
    M[1] *= 1e-30                      # below eps: stays small
    M[2] *= np.float32(1e36)           # squares past float32
    M[4, 3, 5] = np.nan
    M[5, 7, 1] = np.inf
    out = dp.orthogonalize(torch.from_numpy(M).cuda()).cpu().numpy()
    assert np.count_nonzero(out[0]) == 0
    for k in (1, 2, 3):
        ref = optim.newton_schulz(M[k], 5, COEFFS, 1e-7)
        _, bar = _bar(M[3], 5, COEFFS, 1e-7)
        assert np.linalg.norm(out[k] - ref) <= (bar if k != 1 else 1e-25)
    assert np.isnan(out[4]).all() and np.isnan(out[5]).all()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(1, 7), (64, 32), (130, 67), (3, 90, 200), (200, 520), (515, 131)])
def test_optimizer_step(shape, nesterov):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape))
    g, m = (rng.standard_normal(shape).astype(np.float32) * 1e-3 for _ in range(2))
    W = rng.standard_normal(shape).astype(np.float32) * np.float32(0.02)
    lr, beta, wd = 0.05, 0.9, 0.1
    tg, tm, tw = (torch.from_numpy(x.copy()).cuda() for x in (g, m, W))
    dp.muon_step(tg, tm, tw, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd)
    gm, gw = tm.cpu().numpy().astype(np.float64), tw.cpu().numpy().astype(np.float64)
    assert np.array_equal(tg.cpu().numpy(), g)
    flat = lambda x: x.reshape(-1, *shape[-2:])  # noqa: E731
    for k in range(flat(g).shape[0]):
        beta32 = float(np.float32(beta))
        rm, rw, ru = optim.muon_step(flat(g)[k], flat(m)[k], flat(W)[k], lr, beta32, nesterov, wd,
                                     None, 5, COEFFS, 1e-7)
        assert np.abs(flat(gm)[k] - rm).max() <= 2 * U * (np.abs(rm) + np.abs(flat(g)[k])).max()
        u32 = (flat(g)[k] + np.float32(beta) * rm.astype(np.float32)) if nesterov else rm.astype(np.float32)
        ref, bar = _bar(u32, 5, COEFFS, 1e-7)
        # U itself is rounded: what that does to NS(U) is the difference to the reference's
        bar += np.linalg.norm(ref - ru)
        size = lr * np.sqrt(max(1.0, shape[-2] / shape[-1]))
        tol = size * bar + 4 * U * (np.linalg.norm(flat(W)[k]) + size * np.linalg.norm(ru))
        assert np.linalg.norm(flat(gw)[k] - rw) <= tol


def test_optimizer_step_scale_and_repeat():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(9)
    g = torch.from_numpy(rng.standard_normal((96, 40)).astype(np.float32)).cuda()
    W = torch.zeros(96, 40, device="cuda")
    m = torch.zeros_like(W)
    dp.muon_step(g, m, W, lr=1.0, beta=0.0, nesterov=False, scale=2.0)
    O = dp.orthogonalize(g)
    assert torch.allclose(W, -2.0 * O, rtol=4 * U, atol=1e-7)
    W2, m2 = torch.zeros_like(W), torch.zeros_like(m)
    dp.muon_step(g, m2, W2, lr=1.0, beta=0.0, nesterov=False, scale=2.0)
    assert torch.equal(W, W2) and torch.equal(m, m2)


# Matrices of at most 96 rows or columns, too long for one workgroup.
@pytest.mark.parametrize("kind", ["full", "lowrank", "spike"])
@pytest.mark.parametrize("shape", [(1, 6000), (6000, 1), (17, 2000), (32, 1409), (1409, 33), (64, 700),
                                   (65, 650), (650, 65), (96, 417), (3001, 96), (90, 8200)])
def test_thin_matrices(shape, kind):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape))
    M = _matrix(rng, *shape, kind)
    for steps, coeffs in ((1, COEFFS), (5, COEFFS), (4, (1.5, -0.5, 0.0))):
        t = torch.from_numpy(M).cuda()
        out = dp.orthogonalize(t, steps=steps, coeffs=coeffs)
        ref, bar = _bar(M, steps, coeffs, 1e-7)
        err = np.linalg.norm(out.cpu().numpy() - ref)
        assert err <= bar, (steps, err, bar)
        assert torch.equal(out, dp.orthogonalize(t, steps=steps, coeffs=coeffs))
        assert torch.equal(out, dp.orthogonalize(t, steps=steps, coeffs=coeffs, out=t))     # in place


@pytest.mark.parametrize("shape", [(70, 900), (900, 40)])
@pytest.mark.parametrize("n", [2, 150])
def test_stacks_of_thin_matrices(n, shape):
    """Each matrix with its own norm; zero, tiny, huge and not finite ones among them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(n)
    M = np.stack([_matrix(rng, *shape, "full") * np.float32(10.0 ** (k % 5)) for k in range(n)])
    if n > 8:
        M[1] = 0.0
        M[2] *= np.float32(1e-27)                 # below eps: stays small
        M[3] *= np.float32(1e36)
        M[4, 3, 5] = np.nan
        M[5, 7, 1] = np.inf
    t = torch.from_numpy(M).cuda()
    out = dp.orthogonalize(t).cpu().numpy()
    for k in range(n):
        if n > 8 and k in (1, 4, 5):
            assert (out[k] == 0).all() if k == 1 else np.isnan(out[k]).all()
            continue
        ref, bar = _bar(M[k], 5, COEFFS, 1e-7)
        assert np.linalg.norm(out[k] - ref) <= bar, k
    if n > 8:
        t16 = t[6:].bfloat16()
        a, b = dp.orthogonalize(t16), dp.orthogonalize(t16.float())
        assert torch.equal(a, b.bfloat16())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(60, 1000), (2000, 17), (3, 96, 500)])
def test_optimizer_step_of_thin_matrices(shape, nesterov):
    test_optimizer_step(shape, nesterov)


def test_thin_matrices_on_streams_in_graphs_and_buffers():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for shape in ((50, 1303), (1303, 50)):
        M = torch.randn(shape, device="cuda")
        ref = dp.orthogonalize(M)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = dp.orthogonalize(M)
        s.synchronize()
        assert torch.equal(ref, other)
        n = M.numel()
        buf = torch.full((n + 512,), 7.0, device="cuda")
        out = buf[256:256 + n].view(shape)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dp.orthogonalize(M, out=out)
        for _ in range(4):
            M.copy_(torch.randn(shape, device="cuda"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            eager = dp.orthogonalize(M)
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
        assert (buf[:256] == 7).all() and (buf[256 + n:] == 7).all()


def test_in_place_streams_and_graphs():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    M = torch.randn(3, 130, 200, device="cuda")
    ref = dp.orthogonalize(M)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = dp.orthogonalize(M)
    s.synchronize()
    assert torch.equal(ref, other)
    out = torch.zeros_like(M)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.orthogonalize(M, out=out)
    for _ in range(4):
        M.copy_(torch.randn(3, 130, 200, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = dp.orthogonalize(M)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    want = dp.orthogonalize(M)
    assert dp.orthogonalize(M, out=M).data_ptr() == M.data_ptr() and torch.equal(M, want)


def test_outputs_stay_inside_their_buffers():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for shape in ((5, 7), (70, 33), (64, 129)):
        n = shape[0] * shape[1]
        bufs = [torch.full((n + 512,), 7.0, device="cuda") for _ in range(3)]
        g, m, w = (b[256:256 + n].view(shape).normal_() for b in bufs)
        dp.muon_step(g, m, w, lr=0.1)
        dp.orthogonalize(m, out=w)
        torch.cuda.synchronize()
        for b in bufs:
            assert (b[:256] == 7).all() and (b[256 + n:] == 7).all()


def test_binding_refuses_bad_arguments():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    M = torch.randn(16, 24, device="cuda")
    N, W = M.clone(), M.clone()
    for bad in (lambda: dp.orthogonalize(M.t()), lambda: dp.orthogonalize(M.half()),
                lambda: dp.orthogonalize(M[0]), lambda: dp.orthogonalize(M.cpu()),
                lambda: dp.orthogonalize(M, steps=0), lambda: dp.orthogonalize(M, steps=33),
                lambda: dp.orthogonalize(M, eps=0.0), lambda: dp.orthogonalize(M, coeffs=(9, 0, 0)),
                lambda: dp.orthogonalize(M, coeffs=(float("nan"), 0, 0)),
                lambda: dp.orthogonalize(M, out=torch.empty(16, 25, device="cuda")),
                lambda: dp.muon_step(M, M, W, lr=0.1), lambda: dp.muon_step(M, N, N, lr=0.1),
                lambda: dp.muon_step(M, N, W, lr=float("inf")),
                lambda: dp.muon_step(M, N, W, lr=0.1, beta=1.0),
                lambda: dp.muon_step(M, N[:8], W, lr=0.1),
                lambda: dp.muon_step(M.bfloat16(), N, W, lr=0.1)):
        with pytest.raises((ValueError, TypeError, dp.DpfError)):
            bad()
