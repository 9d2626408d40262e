"""Masked rows of the norms' and rotation's gradients give 0 whatever the weights hold."""
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("D", [64, 36, 33])
def test_masked_rows_beside_odd_weights(D, value):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for dtype in (torch.bfloat16, torch.float32):
        g = torch.Generator(device="cuda").manual_seed(D)
        q, k, dq, dk = (torch.randn((2, 6, H, D), generator=g, device="cuda").to(dtype) for H in (3, 1, 3, 1))
        w = torch.ones(D, device="cuda")
        w[3] = value
        mask = torch.tensor([[1, 0, 1, 0, 0, 1], [0, 0, 0, 0, 0, 0]], dtype=torch.uint8, device="cuda")
        freqs, amplitude = dp.rotary_frequencies(D // 2 * 2)
        kw = dict(freqs=freqs, amplitude=amplitude, mask=mask)
        y = dp.qk_norm_rotary(q, k, w, w, **kw)
        r = dp.qk_norm_rotary_backward(dq, dk, q, k, w, w, **kw)
        torch.cuda.synchronize()
        off = mask == 0
        for x in (*y, r.dq, r.dk):
            zeros = bool((x[off] == 0).all())
            assert zeros
        nothing = not bool(r.dq_weight[1].any() or r.dk_weight[1].any())
        assert nothing
