"""The tiled products of the orthogonalised update: every kernel, orientation and form.

Bar as in tests/test_gpu_ortho.py: four times the error e32 of the same iteration in plain
float32 products, plus 8 u ||X||_F, u = 2^-24.
"""
import numpy as np
import pytest

from oracle import optim
from tests.gpu_helpers import need_gpu
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
COEFFS = (3.4445, -4.7750, 2.0315)


def _f32(coeffs):
    return tuple(float(np.float32(x)) for x in coeffs)


def _matrix(rng, R, C, kind):
    if kind == "lowrank":
        k = max(1, min(R, C) // 4)
        M = rng.standard_normal((R, k)) @ rng.standard_normal((k, C)) + 1e-2 * rng.standard_normal((R, C))
    else:
        M = rng.standard_normal((R, C))
    return (M * 1e-3).astype(np.float32)


def _bar(M, steps, coeffs, eps=1e-7):
    ref = optim.newton_schulz(M, steps, _f32(coeffs), eps)
    plain = optim.newton_schulz(M, steps, _f32(coeffs), eps, np.float32).astype(np.float64)
    return ref, 4 * np.linalg.norm(plain - ref) + 8 * U * np.linalg.norm(ref)


# c so small that b / 2c is far above A's eigenvalues, of either sign, near nothing, and b^2 / 4c
# far above a; the usual sets beside them.
@pytest.mark.parametrize("coeffs", [(1.5, -0.625, 0.125), (1.5, -0.5, 0.05), (1.5, -0.5, 0.01), (1.5, -0.5, 1e-3),
                                    (1.5, -0.5, 1e-4), (1.5, -0.5, -1e-5), (1.5, -0.5, 2e-6),
                                    (1.5, -0.5, 1e-30), (1.5, -0.5, 1e-42), (0.2, 1.5, -0.7),
                                    (2.0, -1.5, 0.5), (1.875, -1.25, 0.375), COEFFS])
@pytest.mark.parametrize("kind", ["full", "lowrank"])
@pytest.mark.parametrize("shape", [(160, 200), (330, 140)])
def test_every_size_of_the_last_coefficient(shape, kind, coeffs):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    M = _matrix(np.random.default_rng(sum(shape)), *shape, kind)
    for steps in (1, 5):
        out = dp.orthogonalize(torch.from_numpy(M).cuda(), steps=steps, coeffs=coeffs).cpu().numpy()
        ref, bar = _bar(M, steps, coeffs)
        err = np.linalg.norm(out - ref)
        assert err <= bar, (steps, err / bar)


def test_small_last_coefficient_below_eps_and_in_stacks():
    """Matrices kept at another scale, a zero and a NaN among them."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(8)
    M = np.stack([_matrix(rng, 150, 190, "full") for _ in range(4)])
    M[1] *= np.float32(1e-27)
    M[2] = 0.0
    M[3, 4, 5] = np.nan
    out = dp.orthogonalize(torch.from_numpy(M).cuda(), coeffs=(1.5, -0.5, 1e-4)).cpu().numpy()
    for k in (0, 1):
        ref, bar = _bar(M[k], 5, (1.5, -0.5, 1e-4))
        assert np.linalg.norm(out[k] - ref) <= bar
    assert np.count_nonzero(out[2]) == 0 and np.isnan(out[3]).all()


def _tiles(tile):
    """The "ortho_tile" option for the time of a block."""
    import contextlib

    import sample_gradient_clipping_amd as dp

    @contextlib.contextmanager
    def scope():
        dp.set_option("ortho_tile", tile)
        try:
            yield
        finally:
            dp.set_option("ortho_tile", 0)
    return scope()


# 256: several tiles each way, sizes that are no multiple of it, rows that are no multiple of 4
@pytest.mark.parametrize("coeffs", [COEFFS, (1.5, -0.5, 0.0), (1.5, -0.5, 1e-3)])
@pytest.mark.parametrize("shape", [(300, 200), (200, 300), (257, 701), (701, 257), (520, 512), (130, 1301),
                                   (1301, 131), (3, 270, 330), (3, 330, 270)])
def test_tiles_of_256(shape, coeffs):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(sum(shape))
    flat = [_matrix(rng, *shape[-2:], "full") for _ in range(shape[0] if len(shape) == 3 else 1)]
    M = np.stack(flat).reshape(shape)
    with _tiles(256):
        t = torch.from_numpy(M).cuda()
        out = dp.orthogonalize(t, coeffs=coeffs)
        assert torch.equal(out, dp.orthogonalize(t, coeffs=coeffs))
        assert torch.equal(out, dp.orthogonalize(t, coeffs=coeffs, out=t))
    got = out.cpu().numpy().reshape(-1, *shape[-2:])
    for k, m in enumerate(flat):
        ref, bar = _bar(m, 5, coeffs)
        err = np.linalg.norm(got[k] - ref)
        assert err <= bar, (k, err / bar)


def test_the_option_sets_the_tiles():
    """Seen by the workspace: a pair of halves per element of X twice and of A and B, padded to tiles."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    M = torch.randn(130, 1301, device="cuda")
    for tile in (128, 256):
        with _tiles(tile):
            dp.orthogonalize(M)
        r, c = -(-130 // tile) * tile, -(-1301 // tile) * tile
        pairs = 2 * 4 * (r * c + r * r)
        # beside them the norms' parts, and 64 KB per part of a shared tile of 128
        assert pairs <= dp.get_option("workspace_call_bytes") < pairs + (1 << 16) + (tile == 128) * (1 << 25)


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("shape", [(300, 201), (131, 520), (520, 131)])
def test_bf16_on_either_tile(shape, tile):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(5)
    M = f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))
    t = torch.from_numpy(M.view(np.int16)).view(torch.bfloat16).cuda()
    wide = torch.from_numpy(bf16_bits_to_f32(M)).cuda()
    with _tiles(tile):
        a = dp.orthogonalize(t).view(torch.int16).cpu().numpy().view(np.uint16)
        b = dp.orthogonalize(wide).cpu().numpy()
    assert np.array_equal(a, f32_to_bf16_bits(b))
    ref, bar = _bar(bf16_bits_to_f32(M), 5, COEFFS)
    assert np.linalg.norm(b - ref) <= bar


def _step(torch, dp, rng, shape, nesterov):
    g, m = (rng.standard_normal(shape).astype(np.float32) * 1e-3 for _ in range(2))
    W = rng.standard_normal(shape).astype(np.float32) * np.float32(0.02)
    lr, beta, wd = 0.05, 0.875, 0.1
    tg, tm, tw = (torch.from_numpy(x.copy()).cuda() for x in (g, m, W))
    dp.muon_step(tg, tm, tw, lr=lr, beta=beta, nesterov=nesterov, weight_decay=wd)
    gm, gw = tm.cpu().numpy().astype(np.float64), tw.cpu().numpy().astype(np.float64)
    rm, rw, ru = optim.muon_step(g, m, W, lr, beta, nesterov, wd, None, 5, _f32(COEFFS), 1e-7)
    assert np.abs(gm - rm).max() <= 2 * U * (np.abs(rm) + np.abs(g)).max()
    u32 = (g + np.float32(beta) * rm.astype(np.float32)) if nesterov else rm.astype(np.float32)
    ref, bar = _bar(u32, 5, COEFFS)
    bar += np.linalg.norm(ref - ru)                # what the rounding of U does to NS(U)
    size = lr * np.sqrt(max(1.0, shape[-2] / shape[-1]))
    tol = size * bar + 4 * U * (np.linalg.norm(W) + size * np.linalg.norm(ru))
    assert np.linalg.norm(gw - rw) <= tol


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(300, 202), (131, 523), (780, 260)])
def test_optimizer_step_on_tiles_of_256(shape, nesterov):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    with _tiles(256):
        _step(torch, dp, np.random.default_rng(sum(shape)), shape, nesterov)


@pytest.mark.parametrize("shape", [(301, 200), (140, 390)])
def test_more_tiles_of_128_than_compute_units(shape):
    """Every product of the stack on the kernel for two workgroups per compute unit."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    least = (-(-min(shape) // 128)) * (-(-min(shape) // 128) + 1) // 2     # of the symmetric products
    n = cus // least + 1
    rng = np.random.default_rng(n)
    few = [_matrix(rng, *shape, "full") for _ in range(5)]
    M = np.stack([few[k % 5] * np.float32(1 + k % 7) for k in range(n)])
    with _tiles(128):
        t = torch.from_numpy(M).cuda()
        out = dp.orthogonalize(t)
        assert torch.equal(out, dp.orthogonalize(t))
        out = out.cpu().numpy()
    bars = [_bar(m, 5, COEFFS) for m in few]
    for k in range(n):
        ref, bar = bars[k % 5]
        assert np.linalg.norm(out[k] - ref) <= bar, k


def _bar_on_device(torch, M, steps, coeffs):
    """As _bar, both iterations on the device."""
    a, b, c = _f32(coeffs)

    def iterate(X):
        X = X / torch.sqrt((X.double() ** 2).sum()).to(X.dtype)
        flip = X.shape[0] > X.shape[1]
        X = X.t().contiguous() if flip else X
        for _ in range(steps):
            A = X @ X.t().contiguous()
            X = a * X + (b * A + c * (A @ A)) @ X
        return X.t() if flip else X
    ref, plain = iterate(M.double()), iterate(M.float())
    return ref, float(4 * (plain.double() - ref).norm() + 8 * U * ref.norm())


@pytest.mark.parametrize("shape", [(4096, 4096), (5120, 4096), (12, 768, 768)])
def test_sizes_of_large_layers(shape):
    """Without the option: 4096 x 4096 is where 256-wide tiles start to be the faster ones."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    g = torch.Generator(device="cuda").manual_seed(2)
    M = torch.randn(shape, generator=g, device="cuda") * 1e-3
    out = dp.orthogonalize(M)
    for k in range(shape[0] if len(shape) == 3 else 1):
        m, o = (M[k], out[k]) if len(shape) == 3 else (M, out)
        ref, bar = _bar_on_device(torch, m, 5, COEFFS)
        err = float((o.double() - ref).norm())
        assert err <= bar, err / bar


def test_update_size_of_zero():
    """scale 0 is a step of size 0, not the default one: the momentum moves, the weight decays."""
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(11)
    for shape in ((40, 24), (90, 900), (200, 180)):          # one workgroup, strips, tiles
        g, m, w = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda() for _ in range(3))
        m0, w0 = m.clone(), w.clone()
        dp.muon_step(g, m, w, lr=0.5, beta=0.5, weight_decay=0.5, scale=0.0)
        assert torch.equal(w, w0 * 0.75)
        assert torch.equal(m, m0 * 0.5 + g)
        for bad in (-1.0, -1e-30, float("-inf")):
            with pytest.raises(dp.DpfError):
                dp.muon_step(g, m, w, lr=0.5, scale=bad)
        assert torch.equal(w, w0 * 0.75)
