"""examples/train_bigram.py with its layer: embedding, layer norm, E4M3 linear layer
and head together, gradients of one step against 64-bit arithmetic, and a run."""
import math
import os
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_bigram  # noqa: E402

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def _value(codes, grid):
    n, d = codes.shape
    up = grid.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :d]
    return codes.contiguous().view(E4M3).to(torch.float64) * up


@pytest.mark.parametrize("tied", [False, True])
def test_one_step(tied):
    """Each gradient is that of the values the layer used: rounded to bf16 between
    operators (2^-8 each) and, what the products take, to E4M3 (2^-4 of each element
    of dout, independent of each other, which sums over 500 tokens or 160 columns
    average out).  E4M3 values are read back, so that what remains is bf16 of four
    tensors on the way and sums: within 2^-5 of each gradient's norm; through the
    quantized dout, half a step of 2^-4 of each element: 2^-4 and that."""
    torch.manual_seed(1)
    vocab, dim, n = 700, 160, 500
    m = train_bigram.Bigram(vocab, dim, n, tied, layer=True)
    m.params[0].add_(0.1 * torch.randn(dim, device="cuda"))
    m.params[1].add_(0.1 * torch.randn(dim, device="cuda"))
    tokens, targets = next(train_bigram.batches(vocab, n, 3))
    targets[5] = -1
    w = [_value(c, g) for c, g in zip(m.fp8, m.grid)]
    before = [p.clone() for p in m.params]
    loss = m.step(tokens, targets)
    gamma, beta = (p.double() for p in before)
    h = m.hidden.double()
    c = h - h.mean(1, keepdim=True)
    r = ((c ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5
    y = c * r * gamma + beta
    assert float((m.normed.double() - y).norm()) <= 2.0 ** -8 * float(y.norm())
    x = _value(m.codes_in, m.grid_in)
    assert float((x - y).norm()) <= (2.0 ** -4 + 2.0 ** -8) * float(y.norm())
    out = x @ w[-1].t()
    assert float((m.out.double() - out).norm()) <= 2.0 ** -8 * 1.1 * float(out.norm())
    z = m.out.double() @ w[m.head].t()
    keep = targets >= 0
    logp = torch.log_softmax(z, 1)
    want = torch.where(keep, -logp.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    assert abs(float(loss) - float(want.mean())) < 1e-5 * abs(float(want.mean())) + 1e-6
    dz = logp.exp()
    dz.scatter_add_(1, targets.clamp(min=0)[:, None], -torch.ones(n, 1, dtype=torch.float64, device="cuda"))
    dz *= (keep.double() / n)[:, None]
    dout = dz @ w[m.head]
    quantized = _value(m.codes_out, m.grid_out)
    assert float((m.dout.double() - dout).norm()) <= 2.0 ** -6 * float(dout.norm())
    assert float((quantized - m.dout.double()).norm()) <= 2.0 ** -4 * float(dout.norm())
    dw = quantized.t() @ x
    dn = quantized @ w[-1]
    hat = c * r
    g = dn * gamma
    dh = r * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    grads = [torch.zeros_like(v) for v in w]
    grads[-1] += dw
    grads[m.head] += dz.t() @ m.out.double()
    grads[0].index_add_(0, tokens, dh * dim ** 0.5)
    for got, want in zip(m.grads + m.param_grads, grads + [(dn * hat).sum(0), dn.sum(0)]):
        assert float((got.double() - want).norm()) <= 2.0 ** -5 * float(want.norm())
    norm = math.sqrt(sum(float((v.double() ** 2).sum()) for v in m.grads + m.param_grads))
    assert abs(float(m.norm) - norm) <= 2.0 ** -22 * norm
    # the norm's parameters: one step of the list from zero states
    other = bfz.AdamWList([p.clone() for p in before], *bfz.adamw_states(before, bits=8), grads=m.param_grads)
    other.step(dict(lr=m.lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, step=1), grad_scale=m.coef)
    assert all(torch.equal(a, b) for a, b in zip(other.params, m.params))


def test_it_runs():
    model, losses = train_bigram.train(steps=5, verbose=False, layer=True)
    assert all(math.isfinite(v) for v in losses) and all(bool(p.isfinite().all()) for p in model.params)
