"""Layer norm and its gradient on the GPU against the formulas in 64 bits.

Tolerances (u = 2^-24), with d columns and sums in trees or chains of at most
32 + 20 steps for a row (a thread adds up to 32, the tree the rest):
  mean: 52 u mean|x|;  x - mean: that and u |x - mean|
  rstd: half the relative error of the variance, which the mean's error enters
      squared and every deviation's error (52 u mean|x| + u |x - mean|) twice
  out: (x - mean) rstd weight + bias, four roundings
  dx: sums of g and g h with their terms' errors; dweight, dbias: sums over n rows."""
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: U, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}
STEPS = 52


def _say(*a):
    print("[gpu-layer-norm]", *a, flush=True)
    sys.stdout.flush()


class Exact:
    def __init__(self, x, w, b, eps):
        self.x = x.double()
        self.w = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double()
        self.b = torch.zeros_like(self.w) if b is None else b.double()
        self.mean = self.x.mean(1)
        c = self.x - self.mean[:, None]
        var = (c ** 2).mean(1)
        self.rstd = (var + eps) ** -0.5
        self.h = c * self.rstd[:, None]
        self.out = self.h * self.w + self.b
        # errors
        self.e_mean = STEPS * U * self.x.abs().mean(1)
        self.e_c = self.e_mean[:, None] + U * c.abs()
        e_var = self.e_mean ** 2 + 2 * (self.e_c * c.abs()).mean(1) + (self.e_c ** 2).mean(1) + (STEPS + 4) * U * (var + eps)
        self.e_rstd = self.rstd * (0.6 * e_var / (var + eps) + 4 * U)
        self.e_h = self.e_c * (self.rstd + self.e_rstd)[:, None] + c.abs() * self.e_rstd[:, None] + U * self.h.abs()
        self.e_out = self.e_h * self.w.abs() + 2 * U * (self.out.abs() + (self.h * self.w).abs())

    def grads(self, dy):
        dy = dy.double()
        n, d = dy.shape
        g = dy * self.w
        m1, m2 = g.mean(1, keepdim=True), (g * self.h).mean(1, keepdim=True)
        r = self.rstd[:, None]
        dx = r * (g - m1 - self.h * m2)
        e_g = U * g.abs()
        e_m1 = (STEPS + 1) * U * g.abs().mean(1, keepdim=True)
        e_m2 = ((STEPS + 3) * U * (g * self.h).abs() + g.abs() * self.e_h).mean(1, keepdim=True)
        inner = (g.abs() + m1.abs() + (self.h * m2).abs())
        e_in = e_g + e_m1 + self.e_h * m2.abs() + (self.h.abs() + self.e_h) * e_m2 + 4 * U * inner
        e_dx = (r + self.e_rstd[:, None]) * e_in + inner * self.e_rstd[:, None] + U * dx.abs()
        dw, db = (dy * self.h).sum(0), dy.sum(0)
        # a column's sum: chains over the rows of a workgroup, then over workgroups
        steps = min(n, 200 + n / 256)
        e_dw = ((steps + 3) * U * (dy * self.h).abs() + dy.abs() * self.e_h).sum(0)
        e_db = steps * U * dy.abs().sum(0)
        return (dx, e_dx), (dw, e_dw), (db, e_db)


def near(got, want, e, base=None):
    if base is not None:
        want, e = want + base.double(), e + U * (want.abs() + base.double().abs())
    t = got.dtype
    tol = e * 1.01 + HALF[t] * (want.abs() + e) * 1.0001 + TINY[t]
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


CASES = [(1, 1), (1, 4096), (2, 7), (5, 64), (300, 129), (1000, 1001), (7, 1024), (4, 1025), (600, 2048), (33, 4096), (3, 5000), (70, 8192), (3, 12289), (2, 32768),
         (2500, 96), (9, 20000)]


def _case(n, d, dtype, param):
    torch.manual_seed(n + d)
    x = (torch.randn(n, d, device="cuda") * 2 + torch.randn(n, 1, device="cuda")).to(dtype)
    w, b = (1 + 0.2 * torch.randn(d, device="cuda")).to(param), (0.1 * torch.randn(d, device="cuda")).to(param)
    dy = (torch.randn(n, d, device="cuda") * torch.exp(torch.randn(n, 1, device="cuda"))).to(dtype)
    return x, w, b, dy


def _run(x, w, b, dy, out_type=None, dx_type=None, dp_type=F32, base=None, eps=1e-5):
    n, d = x.shape
    nan = lambda *s, t=F32: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    out, mean, rstd = nan(n, d, t=out_type or x.dtype), nan(n), nan(n)
    bfz.layer_norm(x, w, b, out, eps=eps, mean=mean, rstd=rstd)
    work = bfz.layer_norm_workspace(n, d)
    work.fill_(0xFF)
    dx = nan(n, d, t=dx_type or x.dtype)
    dw, db = (nan(d, t=dp_type), nan(d, t=dp_type)) if base is None else (base[0].clone(), base[1].clone())
    bfz.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, work, accumulate=base is not None)
    return out, mean, rstd, dx, dw, db


@pytest.mark.parametrize("n,d", CASES)
@pytest.mark.parametrize("dtype,param", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)])
def test_layer_norm(n, d, dtype, param):
    _say(n, d, dtype, param)
    x, w, b, dy = _case(n, d, dtype, param)
    ex = Exact(x, w, b, 1e-5)
    out, mean, rstd, dx, dw, db = _run(x, w, b, dy)
    near(mean, ex.mean, ex.e_mean)
    near(rstd, ex.rstd, ex.e_rstd)
    near(out, ex.out, ex.e_out)
    for got, (want, e) in zip((dx, dw, db), ex.grads(dy)):
        near(got, want, e)


@pytest.mark.parametrize("n,d", [(40, 768), (40, 1001)])
def test_types_and_missing_parts(n, d):
    x, w, b, dy = _case(n, d, F32, F32)
    ex = Exact(x, w, b, 1e-5)
    base = (torch.randn(d, device="cuda").to(BF16), torch.randn(d, device="cuda").to(BF16))
    out, mean, rstd, dx, dw, db = _run(x, w, b, dy, BF16, F16, BF16, base)
    (wdx, edx), (wdw, edw), (wdb, edb) = ex.grads(dy)
    near(out, ex.out, ex.e_out)
    near(dx, wdx, edx)
    near(dw, wdw, edw, base[0])
    near(db, wdb, edb, base[1])
    # no weight, no bias, no statistics
    one = torch.empty(n, d, device="cuda")
    bfz.layer_norm(x, None, None, one)
    plain = Exact(x, None, None, 1e-5)
    near(one, plain.out, plain.e_out)
    bfz.layer_norm(x, w, None, one)
    near(one, (ex.h * ex.w), ex.e_out + U * ex.b.abs() * 4)
    # each result alone
    work = bfz.layer_norm_workspace(n, d)
    for k in range(3):
        got = [torch.full_like(x, float("nan")), torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")]
        want = (wdx, wdw, wdb)[k], (edx, edw, edb)[k]
        args = [g if j == k else None for j, g in enumerate(got)]
        bfz.layer_norm_grad(dy, x, w, mean, rstd, *args, work if k else None)
        near(got[k], *want)
    got = torch.empty_like(x)
    bfz.layer_norm_grad(dy, x, None, mean, rstd, got, None, None, None)
    near(got, *plain.grads(dy)[0])


@pytest.mark.parametrize("d,ld,off", [(1000, 1008, 0), (1000, 1003, 1), (96, 101, 3), (5000, 5008, 8), (30000, 30001, 0)])
def test_strides_and_in_place(d, ld, off):
    n = 23
    x0, w, b, dy0 = _case(n, d, BF16, F32)

    def spread(t):
        buf = torch.full((off + (n + 1) * ld,), 7.0, dtype=BF16, device="cuda")
        v = buf[off:off + n * ld].view(n, ld)
        v[:, :d] = t
        return buf, v[:, :d]

    ex = Exact(x0, w, b, 1e-5)
    xb, x = spread(x0)
    ob, out = spread(torch.zeros_like(x0))
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    bfz.layer_norm(x, w, b, out, mean=mean, rstd=rstd)
    near(out, ex.out, ex.e_out)
    db_, dy = spread(dy0)
    gb, dx = spread(torch.zeros_like(x0))
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    work = bfz.layer_norm_workspace(n, d)
    bfz.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, work)
    for got, (want, e) in zip((dx, dw, db), ex.grads(dy0)):
        near(got, want, e)
    for buf in (ob, gb, xb, db_):
        rest = buf.clone()
        rest[off:off + n * ld].view(n, ld)[:, :d] = 7.0
        assert bool((rest == 7.0).all())
    keep_out, keep_dx = out.clone(), dx.clone()
    bfz.layer_norm_grad(dy, x, w, mean, rstd, dy, dw, db, work)  # dx over dout
    assert torch.equal(dy, keep_dx)
    bfz.layer_norm(x, w, b, x)
    assert torch.equal(x, keep_out)


def test_rows_of_extremes():
    """Constant rows (variance 0), a large common offset, huge and tiny values;
    a NaN or infinity stays in its row."""
    d = 700
    x, w, b, dy = _case(9, d, F32, F32)
    x[0] = 3.0
    x[1] = 0.0
    x[2] += 1000.0
    x[3] *= 1e15
    x[4] *= 1e-15
    ex = Exact(x, w, b, 1e-5)
    out, mean, rstd, dx, dw, db = _run(x, w, b, dy)
    near(out, ex.out, ex.e_out)
    near(rstd, ex.rstd, ex.e_rstd)
    near(dx, *ex.grads(dy)[0])
    y = x.clone()
    y[5, 7], y[6, 3] = float("nan"), float("inf")
    two = _run(y, w, b, dy)
    keep = [0, 1, 2, 3, 4, 7, 8]
    assert torch.equal(two[0][keep], out[keep]) and torch.equal(two[3][keep], dx[keep])
    assert bool(two[0][5:7].isnan().all())


def test_no_rows():
    d = 100
    e = torch.empty(0, d, device="cuda")
    v = torch.empty(0, device="cuda")
    w = torch.ones(d, device="cuda")
    bfz.layer_norm(e, w, w, e.clone(), mean=v, rstd=v)
    dw, db = torch.full((d,), 3.0, device="cuda"), torch.full((d,), 4.0, device="cuda")
    work = bfz.layer_norm_workspace(0, d)
    bfz.layer_norm_grad(e, e, w, v, v, e.clone(), dw, db, work, accumulate=True)
    assert bool((dw == 3).all()) and bool((db == 4).all())
    bfz.layer_norm_grad(e, e, w, v, v, e.clone(), dw, db, work)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradient_against_differences():
    n, d, eps = 6, 50, 1e-5
    x, w, b, dy = _case(n, d, F32, F32)
    _, _, _, dx, dw, db = _run(x, w, b, dy, eps=eps)

    def f(x, w, b):
        c = x.double() - x.double().mean(1, keepdim=True)
        return float((dy.double() * (c / ((c ** 2).mean(1, keepdim=True) + eps).sqrt() * w.double() + b.double())).sum())

    for i, j in ((0, 0), (3, 17), (5, 49)):
        step = torch.zeros(n, d, dtype=torch.float64, device="cuda")
        step[i, j] = 1e-4
        slope = (f(x.double() + step, w, b) - f(x.double() - step, w, b)) / 2e-4
        assert abs(slope - float(dx[i, j])) <= 1e-5 * (1 + abs(slope))  # differences: (1e-4)^2 of the third derivative
    for j in (0, 31):
        step = torch.zeros(d, dtype=torch.float64, device="cuda")
        step[j] = 1e-4
        assert abs((f(x, w.double() + step, b) - f(x, w.double() - step, b)) / 2e-4 - float(dw[j])) <= 1e-5 * (1 + abs(float(dw[j])))
        assert abs((f(x, w, b.double() + step) - f(x, w, b.double() - step)) / 2e-4 - float(db[j])) <= 1e-5 * (1 + abs(float(db[j])))


@pytest.mark.parametrize("n,d", [(3, 4096), (3000, 333), (5000, 1024)])
def test_graphs_streams_and_repeats(n, d):
    x, w, b, dy = _case(n, d, BF16, F32)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    work = bfz.layer_norm_workspace(n, d)
    outs = (out, mean, rstd, dx, dw, db)

    def run():
        bfz.layer_norm(x, w, b, out, mean=mean, rstd=rstd)
        bfz.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, work)

    run()
    first = [z.clone() for z in outs]

    def same():
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        [z.fill_(float("nan")) for z in outs]
        work.fill_(0xFF)

    same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same()
