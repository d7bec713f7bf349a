"""Layer norm of rows on a common offset that dwarfs their spread.

The mean is a binary32 sum, off by up to 52 u mean|x| (u = 2^-24, sums of at most
52 steps), and that error is found again as the mean of the x - mean, d, and taken
off them: what is left of it is the rounding of those differences and of their sum,
    e_c = 2 u (|c| + D) + 53 u (mean|c| + D),  c = x - exact mean,  D = 52 u mean|x|
The variance is the mean of d^2 less the square of d's mean, each off by its own
roundings.  The mean that is kept, and that the gradient subtracts, is rounded
once: u |mean| and what is left of its error."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_layer_norm import F32, STEPS, U, Exact, _say, near

pytestmark = pytest.mark.gpu


class Offset(Exact):
    def __init__(self, x, w, b, eps):
        super().__init__(x, w, b, eps)
        c = (self.x - self.mean[:, None])
        spread = c.abs().mean(1)
        D = STEPS * U * self.x.abs().mean(1)
        e_delta = (STEPS + 1) * U * (spread + D)
        var = (c ** 2).mean(1)
        e_var = (STEPS + 8) * U * (var + D ** 2 + eps) + 2 * D * e_delta + e_delta ** 2
        self.e_rstd = self.rstd * (0.6 * e_var / (var + eps) + 4 * U)
        self.e_mean = U * self.mean.abs() + e_delta
        e_c = 2 * U * (c.abs() + D[:, None]) + e_delta[:, None]
        self.e_out = self._h(c, e_c) * self.w.abs() + 2 * U * (self.out.abs() + (self.h * self.w).abs())
        # the gradient's h, from the mean as it was kept
        self.e_h = self._h(c, self.e_mean[:, None] + U * c.abs())

    def _h(self, c, e_c):
        return e_c * (self.rstd + self.e_rstd)[:, None] + c.abs() * self.e_rstd[:, None] + U * self.h.abs()


@pytest.mark.parametrize("d", [64, 700, 1001, 1544, 4096, 5000, 11008, 20000])
@pytest.mark.parametrize("spread", [0.0, 0.01, 1.0])
def test_offset(d, spread):
    torch.manual_seed(d)
    tops = [177.07, 1643.9, 16321.2, -523.3, 1000.0, 3.1e7, 0.1, 0.0]
    n = 2 * len(tops)
    x = torch.tensor(tops * 2, device="cuda")[:, None] + spread * torch.randn(n, d, device="cuda")
    w, b = 1 + 0.2 * torch.randn(d, device="cuda"), 0.1 * torch.randn(d, device="cuda")
    dy = torch.randn(n, d, device="cuda")
    ex = Offset(x, w, b, 1e-5)
    out, mean, rstd = torch.full_like(x, float("nan")), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    _say("offset", d, spread)
    bfz.layer_norm(x, w, b, out, mean=mean, rstd=rstd)
    near(mean, ex.mean, ex.e_mean)
    near(rstd, ex.rstd, ex.e_rstd)
    near(out, ex.out, ex.e_out)
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    bfz.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, bfz.layer_norm_workspace(n, d))
    for got, (want, e) in zip((dx, dw, db), ex.grads(dy)):
        near(got, want, e)


@pytest.mark.parametrize("d", [100, 3000])
def test_rows_beyond_binary32(d):
    """Rows whose squares overflow have an infinite variance, and so nothing but
    the bias.  Where the sum of a row overflows, x - mean is -inf throughout and its
    square inf: 1 / sqrt is 0, and the row -inf * 0, NaN."""
    x = torch.randn(4, d, device="cuda")
    x[1] *= 1e30
    x[2] = 3e30
    x[3] = 3e38
    b = torch.randn(d, device="cuda")
    out, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    bfz.layer_norm(x, None, b, out, mean=mean, rstd=rstd)
    assert torch.equal(out[1], b) and float(rstd[1]) == 0.0
    assert bool(out[2].isfinite().all())  # the mean may be exact
    assert bool(out[3].isnan().all())
    assert bool(out[0].isfinite().all()) and x.dtype == F32
