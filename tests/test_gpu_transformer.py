"""The transformer example: its private gradients against float64 autograd, row by row, its answers
over a cache against the whole prompt's, and a run of it."""
import importlib.util
import os

import pytest

from tests.gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu

NAMES = ("table", "wqkv", "wo", "w", "q_norm", "k_norm")


def _example():
    path = os.path.join(os.path.dirname(__file__), os.pardir, "examples", "private_transformer.py")
    spec = importlib.util.spec_from_file_location("private_transformer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _logits(model, p, ids, documents, positions, kept):
    """One row's logits in float64; kept: what dropout multiplies its input by."""
    import torch
    Hq, Hkv, D = model["heads"]
    T = ids.shape[0]
    X = p["table"][ids]
    q, k, v = (X @ p["wqkv"].t()).view(T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=1)
    angle = positions.double()[:, None, None] * model["freqs"].cpu()
    n = angle.shape[-1]

    def turned(x, w):
        x = w * x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
        a, b, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin(), rest), -1)
    q, k = turned(q, p["q_norm"]), turned(k, p["k_norm"])
    t = torch.arange(T)
    seen = (documents[:, None] == documents[None, :]) & (t[None, :] <= t[:, None])
    heads = []
    for h in range(Hq):
        s = (q[:, h] @ k[:, h * Hkv // Hq].t()) * D ** -0.5
        heads.append(torch.softmax(s.masked_fill(~seen, -float("inf")), -1) @ v[:, h * Hkv // Hq])
    return (X + (torch.cat(heads, -1) @ p["wo"].t()) * kept) @ p["w"].t()


# float32 throughout: from the table to the logits and back ten products of at most 101 terms, norms
# and rotations among them, each within 101 units of 2^-24 of its operands' magnitudes (6e-5 in
# all); the scores and the logits, below 8, become weights whose relative error is their absolute
# one: 8 * 101 * 2^-24 = 5e-5 each at the very worst.
BAR = 2e-4


@pytest.mark.parametrize("D", [10, 16, 9])
def test_private_gradients_match_autograd(D):
    need_gpu()
    import torch
    import sample_gradient_clipping_amd as dp
    example = _example()
    V, width, B, T, p, C = 101, 24, 5, 13, 0.25, 0.8
    model = example.make_model(V, width, 4, 2, D, seed=3)
    for k in example.NORMS:
        model[k] += 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(5)).cuda()
    batch = example.make_batch(B, T, V, torch.Generator().manual_seed(4))
    grads, norms, out = example.private_gradients(model, batch, C, 0.0, seed=7, p=p, dtype=torch.float32)
    kept = dp.dropout(torch.ones((B, T, width), device="cuda"), p, 7).double().cpu()
    assert 0.05 < float((kept == 0).double().mean()) < 0.5
    ids, targets, documents, positions, weight = (x.cpu() for x in batch)
    sums = {k: torch.zeros(model[k].shape, dtype=torch.float64) for k in NAMES}
    clipped = 0
    for i in range(B):
        w = {k: model[k].double().cpu().requires_grad_(True) for k in NAMES}
        z = torch.log_softmax(_logits(model, w, ids[i], documents[i], positions[i], kept[i]), -1)
        logp = z[torch.arange(T), targets[i]]
        g = dict(zip(NAMES, torch.autograd.grad(-(logp * weight[i].double()).sum(), [w[k] for k in NAMES])))
        norm = sum(float((g[k] ** 2).sum()) for k in NAMES) ** 0.5
        assert abs(float(norms[i]) - norm) <= BAR * norm, f"row {i}"
        clipped += norm > C
        for k in NAMES:
            sums[k] += g[k] * min(1.0, C / norm) / B
    assert clipped
    for k, want in sums.items():
        err = float((grads[k].double().cpu() - want).norm() / want.norm())
        assert err <= BAR, f"{k}: {err}"


def test_cached_tokens_match_the_whole_prompt():
    """A prompt taken at once, in pieces and token by token gives the same logits."""
    need_gpu()
    import torch
    example = _example()
    model = example.make_model(101, 24, 4, 2, 10, seed=3)
    ids = torch.randint(0, 101, (3, 40), generator=torch.Generator().manual_seed(6)).cuda()

    def over(pieces):
        cache = [torch.full((3, 50, 2, 10), float("nan"), device="cuda") for _ in range(2)]
        at = 0
        for n in pieces:
            logits = example.next_logits(model, ids[:, at:at + n], cache, at, torch.float32)
            at += n
        return logits
    whole = over([40])
    cpu = {k: model[k].double().cpu() for k in NAMES}
    want = torch.stack([_logits(model, cpu, i, torch.zeros(40), torch.arange(40), 1.0)[-1] for i in ids.cpu()])
    for logits in (whole, over([1] * 40), over([7, 1, 31, 1])):
        assert float((logits[:, 0].double().cpu() - want).norm() / want.norm()) <= BAR


def test_example_runs():
    need_gpu()
    import math
    losses = _example().train(steps=3, B=16, T=16, V=64, width=32, Hq=2, Hkv=1, D=16, log=lambda line: None)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)
