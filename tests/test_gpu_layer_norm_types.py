"""The gradient of layer norm where dout, x, dx and the parameters differ in type, as
with float32 residuals and bfloat16 gradients.  Tolerances: test_gpu_layer_norm.py."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_layer_norm import BF16, F16, F32, Exact, _say, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [5, 512, 1000, 1001, 4096, 8200, 20003])
@pytest.mark.parametrize("x_type,dout_type,dx_type,param,dparam", [(F32, BF16, F32, F32, F32), (F32, F16, BF16, BF16, F32), (BF16, F32, BF16, F32, BF16),
                                                                   (F16, F32, F32, F16, F16), (BF16, F16, F16, BF16, F32)])
def test_gradient(d, x_type, dout_type, dx_type, param, dparam):
    n, pad = 37, 3  # rows on any element's boundary
    torch.manual_seed(d)

    def rows(t):
        return torch.full((n + 1, d + pad), 7.0, dtype=t, device="cuda")

    xb, db, ob = rows(x_type), rows(dout_type), rows(dx_type)
    x, dy, dx = (z[:n, :d] for z in (xb, db, ob))
    x.copy_(torch.randn(n, d, device="cuda") * 2 + torch.randn(n, 1, device="cuda"))
    dy.copy_(torch.randn(n, d, device="cuda") * torch.exp(torch.randn(n, 1, device="cuda")))
    w = (1 + 0.2 * torch.randn(d, device="cuda")).to(param)
    ex = Exact(x, w, None, 1e-5)
    out, mean, rstd = torch.empty(n, d, dtype=dout_type, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    _say("types", d, x_type, dout_type, dx_type)
    bfz.layer_norm(x, w, None, out, mean=mean, rstd=rstd)
    near(out, ex.out, ex.e_out)
    dw, db_ = torch.empty(d, dtype=dparam, device="cuda"), torch.empty(d, dtype=dparam, device="cuda")
    work = bfz.layer_norm_workspace(n, d)
    bfz.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db_, work)
    for got, (want, e) in zip((dx, dw, db_), ex.grads(dy)):
        near(got.contiguous(), want, e)
    assert bool((ob[n] == 7).all()) and bool((ob[:, d:] == 7).all())
