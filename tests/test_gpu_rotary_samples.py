"""Norm weights' gradients of as many samples as take more than 2^32 threads to add up."""
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


def test_weight_gradients_of_a_million_samples():
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, D, part = (1 << 20) + 5, 128, 4099
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, dq, dk = (torch.randn((B, 1, 1, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    w = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    freqs, amplitude = dp.rotary_frequencies(D)
    at = torch.randint(0, 1000, (B, 1), generator=g, device="cuda")
    kw = dict(freqs=freqs, amplitude=amplitude)
    whole = dp.qk_norm_rotary_backward(dq, dk, q, k, w, w, positions=at, **kw)
    torch.cuda.synchronize()
    for first in (0, B // 2, B - part):
        s = slice(first, first + part)
        small = dp.qk_norm_rotary_backward(dq[s], dk[s], q[s], k[s], w, w, positions=at[s], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a[s], b) for a, b in zip(whole, small)), first
