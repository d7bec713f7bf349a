"""The clipped step on a factor that is not finite: padding stays +0.0, as a
step on gradients multiplied beforehand leaves it."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("factor", [float("nan"), float("inf")])
@pytest.mark.parametrize("dims", [[(2, 130, 257), (1, 129, 200)], [(1, 300, 1000)]])
def test_padding_takes_no_part(factor, dims):
    torch.manual_seed(5)
    plan = bfz.Plan(dims, 3, 2)
    q = plan.shard_tiles
    coef = torch.full((1,), factor, device="cuda")
    grads = [torch.rand(d, device="cuda") + 0.5 for d in dims]
    clipped = [g * coef for g in grads]
    hp = bfz.AdamW(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3)

    def run(kind, gs, **kw):
        st = [torch.zeros(q * 16384, device="cuda") for _ in range(3)]
        codes = torch.zeros(q * 16384, dtype=torch.uint8, device="cuda")
        sc = torch.zeros(q, device="cuda")
        f8 = [torch.zeros(d, dtype=torch.uint8, device="cuda") for d in dims]
        gr = [torch.zeros(E, -(-H // 128), -(-W // 128), device="cuda") for E, H, W in dims]
        t8 = [torch.zeros(E, W, H, dtype=torch.uint8, device="cuda") for E, H, W in dims]
        tg = [torch.zeros(E, W, -(-H // 128), device="cuda") for E, H, W in dims]
        if kind == "fold":
            bfz.fold_adamw_fp8_step(plan, gs, *st, codes, sc, hp, **kw)
        elif kind == "unpack":
            bfz.fold_adamw_fp8_step_unpack(plan, gs, *st, codes, sc, f8, gr, hp, **kw)
        else:
            bfz.fold_adamw_fp8_step_unpack_t(plan, gs, *st, codes, sc, f8, gr, t8, tg, hp, **kw)
        return st + [sc]

    for kind in ("fold", "unpack", "t"):
        for x, y in zip(run(kind, grads, grad_scale=coef), run(kind, clipped)):
            assert torch.equal(torch.isnan(x), torch.isnan(y)), kind
            assert torch.equal(x[~torch.isnan(x)], y[~torch.isnan(y)]), kind
