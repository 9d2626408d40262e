"""The language-model example: its private gradients against float64 autograd, sample by
sample, and a few training steps."""
import importlib.util
import os

import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(__file__), os.pardir, "examples", "private_language_model.py")
    spec = importlib.util.spec_from_file_location("private_language_model", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _expected(model, ids, targets, mask, C):
    """Each sample's gradients by autograd in float64 on the CPU, clipped together, averaged."""
    import torch
    names = ("table", "w1", "w2")
    sums = {k: torch.zeros(model[k].shape, dtype=torch.float64) for k in names}
    norms = []
    for i in range(ids.shape[0]):
        p = {k: model[k].double().cpu().requires_grad_(True) for k in names}
        keep = mask[i].bool().cpu()
        z = torch.relu(p["table"][ids[i].cpu()[keep]] @ p["w1"].t()) @ p["w2"].t()
        loss = torch.nn.functional.cross_entropy(z, targets[i].cpu()[keep])
        g = dict(zip(names, torch.autograd.grad(loss, [p[k] for k in names])))
        norm = sum(float((g[k] ** 2).sum()) for k in names) ** 0.5
        norms.append(norm)
        for k in names:
            sums[k] += g[k] * min(1.0, C / norm)
    return {k: s / ids.shape[0] for k, s in sums.items()}, norms


# float32 throughout: three products of at most 101 terms, each within 101 units of 2^-24 of its
# operands' magnitudes, a softmax of logits below 8 in between (their absolute error becomes the
# probabilities' relative one, 8 * 101 * 2^-24 = 5e-5 at the very worst).
BAR = 1e-4


def test_private_gradients_match_autograd():
    need_gpu()
    import torch
    example = _example()
    V, D, H, B, T = 101, 24, 40, 5, 11
    model = example.make_model(V, D, H, seed=3)
    ids, targets, mask = example.make_batch(B, T, V, torch.Generator().manual_seed(4))
    ids[1, :] = ids[1, 0]                         # one token throughout a sentence
    C = 0.8
    grads, norms, _ = example.private_gradients(model, ids, targets, mask, C, 0.0, seed=0,
                                                dtype=torch.float32)
    want, want_norms = _expected(model, ids, targets, mask, C)
    assert any(n > C for n in want_norms)
    for i, n in enumerate(want_norms):
        assert abs(float(norms[i]) - n) <= BAR * n, f"sample {i}"
    for k, w in want.items():
        err = float((grads[k].double().cpu() - w).norm() / w.norm())
        assert err <= BAR, f"{k}: {err}"


def test_training_lowers_the_loss():
    need_gpu()
    losses = _example().train(steps=12, B=64, T=16, V=64, D=32, H=64, sigma=0.0, log=lambda line: None)
    assert losses[-1] < losses[0]
