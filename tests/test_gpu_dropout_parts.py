"""Dropout from one part of an array's rows into another."""
import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("B,T", [(3, 11), (4, 1), (1, 7)])
def test_input_output_and_residual_are_parts_of_one_array(B, T, D):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    for dtype in (torch.float32, torch.bfloat16):
        rows = torch.randn((B, T, 4 * D), device="cuda").to(dtype)
        x, r, y, rest = rows.split(D, dim=2)
        want = dp.dropout(x.contiguous(), 0.3, 5, 9, residual=r.contiguous())
        kept = [t.clone() for t in (x, r, rest)]
        dp.dropout(x, 0.3, 5, 9, residual=r, out=y)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip((x, r, rest), kept))
        for by in (1, D - 1):           # shares entries with x: refused
            with pytest.raises(dp.DpfError):
                dp.dropout(x, 0.3, 5, 9, out=rows[:, :, by:by + D])
        with pytest.raises(dp.DpfError):
            dp.dropout(x, 0.3, 5, 9, residual=r, out=rows[:, :, 2 * D - 1:3 * D - 1])
