"""A gradient whose square overflows makes its block of 8-bit states NaN, its roots
as well as the others' in the block, and nothing else."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)


@pytest.mark.parametrize("n", [256 * 3, 256 * 20, 256 * 20 + 100])
def test_root_that_overflows(n):
    torch.manual_seed(n)
    p, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    g[300:310] = 0.0

    def step(g):
        q = p.clone()
        m, v, ms, vs = bfz.adamw_states([q], bits=8)
        bfz.AdamWList([q], m, v, ms, vs, grads=[g]).step(HP)
        return [q, m[0], v[0], ms[0], vs[0]]

    first = step(g)
    g[259] = 1e25
    second = step(g)
    q, m, v, ms, vs = second
    root = v.view(E4M3).float() * vs.repeat_interleave(256)[:n]
    assert float(vs[1]) == float("inf") and bool(root[256:512].isnan().all())
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[256:512] = False
    for a, b in zip(first[1:3], second[1:3]):
        assert torch.equal(a[rest], b[rest])
    blocks = [k for k in range(vs.numel()) if k != 1]
    assert torch.equal(first[3][blocks], ms[blocks]) and torch.equal(first[4][blocks], vs[blocks])
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[259] = False
    assert torch.equal(first[0][keep], q[keep]) and bool(ms.isfinite().all())
