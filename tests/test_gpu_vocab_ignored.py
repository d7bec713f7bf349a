"""Tokens without a target whose hidden rows, lse and dloss hold NaN or
infinity: they have no gradient and add none."""
import pytest
import torch

from tests.test_gpu_vocab_loss import _check, _run, _say, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("dw_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(3, 128), (16, 72), (17, 128), (70, 100), (300, 512)])
def test_ignored_tokens_may_hold_anything(n, d, dw_type, kind):
    """A token whose target lies outside the vocabulary has no gradient and adds
    none, whatever its hidden row, its lse and its dloss are."""
    _say("ignored tokens", n, d, kind, dw_type)
    torch.manual_seed(n + d)
    V = 600
    h = torch.randn(n, d, device="cuda").to(torch.bfloat16)
    w, grid, value = _weight(V, d, kind)
    t = torch.randint(0, V, (n,), device="cuda")
    dloss = torch.rand(n, device="cuda") + 0.1
    for k, bad in ((0, float("nan")), (2, float("inf"))):
        t[k] = -1
        h[k, 5:9] = bad
        dloss[k] = bad
    loss, lse, dh, dw = _run(h, w, grid, t, dloss, dw_type)
    assert bool((loss[[0, 2]] == 0).all()) and bool((dh[[0, 2]] == 0).all())
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[0, 2]] = False
    _check(h[keep], value, t[keep], (loss[keep], lse[keep], dh[keep], dw), dloss[keep])
