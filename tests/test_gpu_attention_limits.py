"""Single tokens of many long sequences: more heads times positions than a call of as many queries may
have, against the fp64 oracle for some of the samples.  The keys' memory is one sample's, seen by all."""
import numpy as np
import pytest

from oracle import attention as oracle
from oracle.dp_linear import widen
from tests.gpu_helpers import need_gpu, to_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("Hkv", [8, 1])
def test_single_tokens_of_many_long_sequences(Hkv, masked):
    torch = need_gpu()
    import sample_gradient_clipping_amd as dp
    B, Hq, Tk, D = 64, 64, 65536, 16
    rng = np.random.default_rng(Hkv)
    q, dout = (f32_to_bf16_bits(rng.standard_normal((B, 1, Hq, D)).astype(np.float32)) for _ in range(2))
    k, v = (f32_to_bf16_bits(rng.standard_normal((1, Tk, Hkv, D)).astype(np.float32)) for _ in range(2))
    mask = (rng.random((B, Tk)) < 0.7).astype(np.uint8) if masked else None
    if masked:
        mask[:, -1] = 1
        mask[5, -1] = 0
    tq, tk, tv, td = (to_dev(x, "bf16", torch) for x in (q, k, v, dout))
    tk, tv = (x.expand(B, Tk, Hkv, D) for x in (tk, tv))
    m = None if mask is None else torch.from_numpy(mask).cuda()
    r = dp.attention(tq, tk, tv, mask=m)
    grads = dp.attention_backward(td, tq, tk, tv, r.out, r.lse, mask=m)
    torch.cuda.synchronize()
    for b in (0, 5, 63):
        one = [widen(x, "bf16") for x in (q[b:b + 1], k, v)]
        want = oracle.oracle_attention(*one, None if mask is None else mask[b:b + 1], None, True, D ** -0.5, "bf16",
                                       dout=widen(dout[b:b + 1], "bf16"))
        for name, got, (value, bar) in zip(("out", "lse", "dq", "dk", "dv"), (*r, *grads), want):
            err = np.abs(got[b:b + 1].double().cpu().numpy() - value)
            fine = bool(np.isfinite(err).all() and (err <= bar).all())
            assert fine, (b, name, float(err.max()))
