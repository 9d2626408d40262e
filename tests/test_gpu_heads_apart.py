"""In-place rotation and gradients into parts of one array, in every order of its dimensions and for
single tokens: bitwise what tensors of their own give, and nothing else written."""
import numpy as np
import pytest

from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _parts(torch, layout, B, T, H, D, fill, dtype):
    """An array with room for three parts of H heads (and a guard), and views of it [B, T, H, D]."""
    make = lambda *s: torch.full(s, fill, dtype=dtype, device="cuda")  # noqa: E731
    if layout == "rows":
        rows = make(B, T, 4 * H, D)
        return rows, [rows[:, :, i * H:(i + 1) * H] for i in range(3)]
    if layout == "samples":
        rows = make(B, 4, H, T, D)
        return rows, [rows[:, i].transpose(1, 2) for i in range(3)]
    if layout == "swapped":
        rows = make(T, B, 4, H, D)
        return rows, [rows[:, :, i].transpose(0, 1) for i in range(3)]
    rows = make(B, T, H, 4, D)
    return rows, [rows[:, :, :, i] for i in range(3)]


def _rest(layout, rows, H):
    """The part that no view covers."""
    return {"rows": lambda: rows[:, :, 3 * H:], "samples": lambda: rows[:, 3], "swapped": lambda: rows[:, :, 3],
            "heads": lambda: rows[:, :, :, 3]}[layout]()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["rows", "samples", "swapped", "heads"])
@pytest.mark.parametrize("B,T", [(16, 1), (2, 1), (1, 1), (3, 5), (2, 70)])
@pytest.mark.parametrize("D", [64, 45])
def test_parts_of_one_array(D, B, T, layout, dtype):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    rng = np.random.default_rng(B + T + D)
    H = 2

    def some():
        x = rng.standard_normal((B, T, H, D)).astype(np.float32)
        return to_dev(f32_to_bf16_bits(x) if dtype == "bf16" else x, dtype, torch)
    q, k, v, dout = (some() for _ in range(4))
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda()
    freqs, amplitude = dp.rotary_frequencies(D // 2 * 2)
    kw = dict(freqs=freqs, amplitude=amplitude)
    wq, wk = dp.qk_norm_rotary(q, k, w, w, **kw)
    want = dp.attention(wq, wk, v)
    grads = dp.attention_backward(dout, wq, wk, v, want.out, want.lse)
    norms = dp.qk_norm_rotary_backward(grads[0], grads[1], q, k, w, w, **kw)

    rows, parts = _parts(torch, layout, B, T, H, D, 7.0, q.dtype)
    for p, x in zip(parts, (q, k, v)):
        p.copy_(x)
    dp.qk_norm_rotary(parts[0], parts[1], w, w, **kw, q_out=parts[0], k_out=parts[1])
    drows, dparts = _parts(torch, layout, B, T, H, D, 7.0, q.dtype)
    r = dp.attention(*parts)
    dp.attention_backward(dout, *parts, r.out, r.lse, dq=dparts[0], dk=dparts[1], dv=dparts[2])
    got = [x.clone() for x in dparts]
    n = dp.qk_norm_rotary_backward(dparts[0], dparts[1], q, k, w, w, **kw, dq=dparts[0], dk=dparts[1])
    torch.cuda.synchronize()
    assert torch.equal(parts[0], wq) and torch.equal(parts[1], wk) and torch.equal(parts[2], v)
    assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert all(torch.equal(a, b) for a, b in zip(n, norms))
    assert (_rest(layout, rows, H) == 7.0).all() and (_rest(layout, drows, H) == 7.0).all()
