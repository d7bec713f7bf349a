"""Vocabulary rows whose logits are infinite: -inf adds nothing, +inf makes lse
+inf, as the sums of their exponentials have it."""
import pytest
import torch

from tests.test_gpu_vocab_loss import _check, _run, _say, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [3, 16, 17, 100, 300])
def test_rows_of_minus_infinity(n):
    """Rows struck out with -inf logits, whole tiles of them included, add
    nothing: lse and loss are those of the other rows."""
    _say("-inf rows", n)
    torch.manual_seed(n)
    V, d = 1500, 200
    h = torch.randn(n, d, device="cuda")
    h[:, 0] = h[:, 0].abs() + 0.5
    h = h.to(torch.bfloat16)
    w, _, value = _weight(V, d, "bf16")
    out = torch.zeros(V, dtype=torch.bool, device="cuda")
    out[256:1024] = True  # whole tiles of every width
    out[[0, 3, 1100, 1499]] = True
    w[out] = 0.0
    w[out, 0] = -float("inf")
    left = torch.nonzero(~out)[:, 0]
    t = left[torch.randint(0, len(left), (n,), device="cuda")]
    got = _run(h, w, None, t)
    _check(h, value[left], torch.searchsorted(left, t), got)


@pytest.mark.parametrize("n", [3, 17, 300])
def test_infinite_logits(n):
    """One +inf logit: lse is +inf; none but -inf: lse is -inf."""
    torch.manual_seed(n)
    V, d = 700, 64
    h = torch.ones(n, d, device="cuda").to(torch.bfloat16)
    w, _, _ = _weight(V, d, "bf16")
    t = torch.full((n,), 5, device="cuda")
    w[400] = 0.0
    w[400, 7] = float("inf")
    loss, lse = _run(h, w, None, t)
    assert bool((lse == float("inf")).all()) and bool((loss == float("inf")).all())
    w.zero_()
    w[:, 0] = -float("inf")
    loss, lse = _run(h, w, None, t)
    assert bool((lse == -float("inf")).all())
