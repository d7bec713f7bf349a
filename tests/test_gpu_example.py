"""examples/train_bigram.py: the operators together, one training step checked
against 64-bit arithmetic and a run that has to learn."""
import math
import os
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_bigram  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tied", [False, True])
def test_one_step(tied):
    """Gradients from the FP8 weights' values: hidden is rounded to bf16 by the
    lookup and used as rounded, so what differs from 64 bits is dz in bf16 (2^-8
    of each), sums in binary32 and dhidden in bf16 (2^-8): within 2^-6 of the
    gradient's norm.  The norm is of the gradients as written, the step that
    follows is the library's own on those gradients."""
    torch.manual_seed(1)
    vocab, dim, n = 700, 160, 500
    m = train_bigram.Bigram(vocab, dim, n, tied)
    tokens, targets = next(train_bigram.batches(vocab, n, 3))
    targets[5] = -1
    w = [(c.view(torch.float8_e4m3fn).to(torch.float64) * g.double().repeat_interleave(128, 0)[:vocab].repeat_interleave(128, 1)[:, :dim])
         for c, g in zip(m.fp8, m.grid)]
    before = m.state.clone()
    loss = m.step(tokens, targets)
    h = m.hidden.double()
    assert float((h - w[0][tokens] * dim ** 0.5).abs().max()) <= 2.0 ** -8 * float((w[0].abs().max() * dim ** 0.5)) * 1.01
    z = h @ w[-1].t()
    keep = targets >= 0
    logp = torch.log_softmax(z, 1)
    want = torch.where(keep, -logp.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    assert abs(float(loss) - float(want.mean())) < 1e-5 * abs(float(want.mean())) + 1e-6
    dz = logp.exp()
    dz.scatter_add_(1, targets.clamp(min=0)[:, None], -torch.ones(n, 1, dtype=torch.float64, device="cuda"))
    dz *= (keep.double() / n)[:, None]
    grads = [torch.zeros_like(x) for x in w]
    grads[-1] += dz.t() @ h
    grads[0].index_add_(0, tokens, (dz @ w[-1]) * dim ** 0.5)
    for got, g in zip(m.grads, grads):
        assert float((got.double() - g).norm()) <= 2.0 ** -6 * float(g.norm())
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in m.grads))
    assert abs(float(m.norm) - norm) <= 2.0 ** -23 * norm
    coef = torch.tensor([min(1.0, 1.0 / (norm + 1e-6))], device="cuda")
    assert abs(float(m.coef) - float(coef)) <= 2.0 ** -23
    # the step on gradients clipped beforehand
    other = train_bigram.Bigram(vocab, dim, n, tied)
    other.state.copy_(before)
    for a, b in zip(other.grads, m.grads):
        a.copy_(b * m.coef)
    other._update()
    assert torch.equal(other.state, m.state) and all(torch.equal(a, b) for a, b in zip(other.fp8, m.fp8))


@pytest.mark.parametrize("tied", [False, True])
def test_it_learns(tied):
    """Uniform guessing costs log 1000 = 6.9; the best possible is log 2."""
    _, losses = train_bigram.train(steps=60, tied=tied, verbose=False)
    print("[gpu-example]", "tied" if tied else "untied", losses[0], losses[-1], flush=True)
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.5 * losses[0]
