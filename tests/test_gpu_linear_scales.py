"""Scales far apart, zero, subnormal and NaN, and NaN codes, in all three products and
for results of each type.  Tolerances: those of test_gpu_linear.py for the sums, and
for products of two scales below 2^-126, which keep 2^-149 of themselves at worst, as
much for each of their block's 128 products of at most 448 * 448."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_linear import BF16, F16, F32, HALF, U, _say, _tiny, quantized, value, weight

pytestmark = pytest.mark.gpu
NAN = 0x7F


def near(got, a, b, blocks):
    t = got.dtype
    want, size = a @ b, a.abs() @ b.abs()
    e = (2 * 128 + 2 * blocks + 8) * U * size + blocks * 2.0 ** -149 * 448 * 448 * 128
    if t == BF16:
        e = e + 7 * 2.0 ** -13 * size
    tol = e + HALF[t] * (want.abs() + e) * 1.0001 + _tiny(t)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


def spread(scales, lo, hi):
    """The same scales, powers of two apart."""
    return scales * torch.exp2(torch.randint(lo, hi, scales.shape, device="cuda").float())


# float16 holds results up to 2^16: sums of some 2^11 here, and factors up to 1
RANGE = {F32: (-40, 40), BF16: (-40, 40), F16: (-40, 1)}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [2, 30, 60, 200])
def test_forward(n, dtype):
    torch.manual_seed(n)
    rows, cols = 300, 640
    w, grid, _ = weight(rows, cols, 0.1)
    grid = spread(grid, *RANGE[dtype])
    grid[1, 2], grid[2, 0], grid[0, 4] = 0.0, 2.0 ** -149, 2.0 ** -130
    for tiles in (False, True):
        codes, scales = quantized(torch.randn(n, cols, device="cuda"), tiles)
        scales = spread(scales, -20, 1)
        work = bfz.linear_workspace(n, w)
        out = torch.empty(n, rows, dtype=dtype, device="cuda")
        _say("scales, forward", n, dtype, tiles)
        bfz.linear(codes, w, grid, out, work, scales=scales, tiles=tiles)
        near(out, value(codes, scales, tiles), value(w, grid, True).t(), 5)
        # a NaN code reaches its token, a NaN scale its tokens, a NaN of the weight its column
        codes[0, 70] = NAN
        touched = torch.zeros(n, dtype=torch.bool, device="cuda")
        touched[0] = True
        if tiles:
            scales[-1, 1] = float("nan")
            touched[(n - 1) // 128 * 128:] = True
        else:
            scales[1, n - 1] = float("nan")
            touched[n - 1] = True
        other = w.clone()
        other[131, 5] = NAN
        two = torch.empty_like(out)
        bfz.linear(codes, other, grid, two, work, scales=scales, tiles=tiles)
        assert bool(two[touched].isnan().all()) and bool(two[:, 131].isnan().all())
        two[:, 131] = out[:, 131]
        assert torch.equal(two[~touched], out[~touched])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [2, 60, 300])
def test_gradients(n, dtype):
    torch.manual_seed(n)
    rows, cols = 300, 640
    w, grid, _ = weight(rows, cols, 0.1)
    grid = spread(grid, *RANGE[dtype])
    grid[1, 2], grid[2, 0], grid[0, 4] = 0.0, 2.0 ** -149, 2.0 ** -130
    dc, ds = quantized(torch.randn(n, rows, device="cuda"), True)
    xc, xs = quantized(torch.randn(n, cols, device="cuda"), True)
    ds, xs = spread(ds, -20, 1), spread(xs, *RANGE[dtype])
    ds[0, 1], xs[0, 2], xs[0, 3] = 2.0 ** -149, 0.0, 2.0 ** -130
    work = bfz.linear_workspace(n, w)
    dx, dw = torch.empty(n, cols, dtype=dtype, device="cuda"), torch.empty(rows, cols, dtype=dtype, device="cuda")
    _say("scales, gradients", n, dtype)

    def run(dc, ds, xc, xs, w, grid):
        bfz.linear_grad_input(dc, w, grid, dx, work, scales=ds, tiles=True)
        bfz.linear_grad_weight(dc, ds, xc, xs, dw, work)
        return dx.clone(), dw.clone()

    first = run(dc, ds, xc, xs, w, grid)
    near(first[0], value(dc, ds, True), value(w, grid, True), 3)
    near(first[1], value(dc, ds, True).t(), value(xc, xs, True), -(-n // 128))
    # a NaN code of dout: its token of dx, its row of dweight; of the weight: its
    # column of dx; of x: its column of dweight
    dc[1, 7], xc[0, 500], w[299, 33] = NAN, NAN, NAN
    second = run(dc, ds, xc, xs, w, grid)
    assert bool(second[0][1].isnan().all()) and bool(second[0][:, 33].isnan().all())
    assert bool(second[1][7].isnan().all()) and bool(second[1][:, 500].isnan().all())
    second[0][1], second[0][:, 33] = first[0][1], first[0][:, 33]
    second[1][7], second[1][:, 500] = first[1][7], first[1][:, 500]
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    # a NaN scale of dout's tile: its tokens, its rows of dweight
    dc[1, 7] = xc[0, 500] = w[299, 33] = 0
    first = run(dc, ds, xc, xs, w, grid)
    ds[0, 2] = float("nan")
    second = run(dc, ds, xc, xs, w, grid)
    assert bool(second[0][:128].isnan().all()) and torch.equal(second[0][128:], first[0][128:])
    assert bool(second[1][256:].isnan().all()) and torch.equal(second[1][:256], first[1][:256])
