"""A float32 dweight has more bits than a bf16 dz could give it.

dz goes to the matrix cores as two bf16 parts, off by 2^-8 * 2^-8 of itself
together (half a step of each).  Beside that stands p's own error: the logits'
and lse's binary32 sums ((d + d/64 + 4) u sum|h w|, as in test_gpu_vocab_loss.py)
and exponentials of arguments of up to 64 + 1.45 |z - lse|, rounded once.  With
`rounded` the parts are one, 2^-8."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_vocab_loss import U, _case, _say

pytestmark = pytest.mark.gpu


def _limits(h, value, t, dloss, parts):
    n, d = h.shape
    V = value.shape[0]
    hd = h.double()
    z = hd @ value.t()
    ez = ((d + d / 64 + 4) * U * (hd.abs() @ value.abs().t())).amax(1)
    keep = (t >= 0) & (t < V)
    tt = t.clamp(0, V - 1).long()
    lse = torch.logsumexp(z, 1)
    span = (z - lse[:, None]).abs().amax(1)
    elog = ez + (4 * span + 8 + 48 + V / 2048) * U + 4 * U * lse.abs()
    up = torch.where(keep, dloss.double(), 0.0)
    p = (z - lse[:, None]).exp() * up[:, None]
    ep = p.abs() * (ez + elog + (64 + 1.45 * span) * U + 8 * U)[:, None]
    dz = p.scatter_add(1, tt[:, None], -up[:, None])
    edz = 2.0 ** (-8 * parts) * dz.abs() + 1.01 * ep + 2.0 ** -133
    want = dz.t() @ hd
    return want, edz.t() @ hd.abs() + (2 * n + 4) * U * (dz.abs().t() @ hd.abs()) + U * want.abs()


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,V,d", [(1, 300, 64), (5, 257, 100), (16, 5000, 200), (17, 600, 136), (130, 513, 1000), (512, 4000, 128), (2050, 3001, 328)])
def test_float32_dweight(n, V, d, kind, constant):
    _say("f32 dweight", n, V, d, kind, constant)
    h, w, grid, value, t = _case(n, V, d, kind)
    dloss = torch.full((n,), 1.0 / n, device="cuda") if constant else torch.rand(n, device="cuda") + 0.1
    work = bfz.vocab_loss_workspace(n, V, d, weight_dtype=w.dtype)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    bfz.vocab_loss(h, w, t, loss, lse, work, grid=grid)
    got = {}
    for rounded in (False, True):
        work.fill_(0xFF)
        dw = got[rounded] = torch.full((V, d), float("nan"), device="cuda")
        dh = torch.empty_like(h)
        bfz.vocab_loss_grad(h, w, t, lse, dloss, dh, dw, work, grid=grid, rounded=rounded)
        want, limit = _limits(h, value, t, dloss, 1 if rounded else 2)
        bad = ~((dw.double() - want).abs() <= limit)
        assert not bool(bad.any()), (rounded, int(bad.sum()), dw[bad][:4], want[bad][:4], limit[bad][:4])
        again = torch.full_like(dw, float("nan"))
        bfz.vocab_loss_grad(h, w, t, lse, dloss, None, again, work, grid=grid, rounded=rounded)
        assert torch.equal(dw, again)
        base = torch.randn(V, d, device="cuda")
        both = base.clone()
        bfz.vocab_loss_grad(h, w, t, lse, dloss, None, both, work, grid=grid, rounded=rounded, accumulate=True)
        bad = (both.double() - base.double() - want).abs() > limit + U * (base.double() + want).abs() * 1.01
        assert not bool(bad.any())
    off = {k: float((x.double() - want).norm() / want.norm()) for k, x in got.items()}
    _say("relative error", off)
    assert off[False] <= 1e-5


def test_rounded_is_of_float32_only():
    h, w, grid, value, t = _case(20, 300, 64, "bf16")
    work = bfz.vocab_loss_workspace(20, 300, 64, weight_dtype=w.dtype)
    x = torch.zeros(20, device="cuda")
    with pytest.raises(ValueError):
        bfz.vocab_loss_grad(h, w, t, x, x, None, torch.zeros_like(w), work, rounded=True)
