"""Every form in which the linear layer's products are launched: tiles, waves, splits
and half-wide last tiles, in each product and for results of each type, within larger
buffers.  Tolerances are those of test_gpu_linear.py."""
import ctypes as C

import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_linear import BF16, F16, F32, _say, check, quantized, value, weight

CODE = {F32: 0, BF16: 1, F16: 2}

# (rows of the result, elements of each, length of the sum)
SIZES = [(652, 5499, 262), (5458, 258, 257), (2844, 136, 4099), (2755, 143, 5662), (74, 79, 266), (74, 77, 1079), (74, 74, 1886), (1834, 5923, 265),
         (6982, 1560, 263), (5393, 1303, 270), (6063, 801, 257), (5033, 3088, 259)]
FEW = [(1, 300, 640), (16, 4300, 260), (17, 130, 200), (32, 4999, 300), (40, 3000, 513), (64, 5001, 257), (50, 8209, 300)]


def dims(product, across, m, k):
    """(n, rows, cols) of the product whose result is across x m."""
    return ((across, m, k), (across, k, m), (k, across, m))[product]


def form(product, n, rows, cols, dtype):
    out = (C.c_int64 * 6)()
    assert bfz.lib().bfz_linear_shape(product, n, rows, cols, CODE[dtype], out) == 0
    tm, tn, waves, splits, whole, exact = out
    across = rows if product == 2 else n
    return tm, tn, waves, splits > 1, whole < across, bool(exact)


@pytest.mark.parametrize("product", [0, 1, 2])
def test_sizes_reach_every_form(product):
    """(CPU) The forms that the sizes below launch are all that there are: tiles of
    128 with and without splits, of 256 with and without half-wide last ones."""
    cut = [(128, 64, 8), (128, 128, 8)]
    for dtype in (F32, BF16, F16):
        exact = dtype != BF16
        want = {(*c, split, False, exact) for c in cut for split in (False, True)} | {(128, 128, 4, False, False, exact)}
        for wide in (128,) if exact else (128, 256):
            want |= {(256, wide, 8, False, half, exact) for half in (False, True)}
        assert {form(product, *dims(product, *s), dtype) for s in SIZES} == want
    few = {form(0, *s, t) for s in FEW for t in (F32, BF16)}
    want = {(tm, tn, 8, False, False, True) for tm, tn in ((16, 16), (32, 16), (16, 32), (32, 32), (16, 64), (32, 64), (48, 64))}
    assert few == want | {(*w[:5], False) for w in want if w[1] > 16}


def inside(rows, cols, dtype):
    """A result of NaNs in a larger buffer of nines."""
    buf = torch.full((rows + 1, cols + 3), 9.0, dtype=dtype, device="cuda")
    out = buf[:rows, :cols]
    out.fill_(float("nan"))
    return buf, out


def untouched(buf, rows, cols):
    return bool((buf[rows] == 9).all()) and bool((buf[:, cols:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("product", [0, 1, 2])
def test_form(product, size):
    n, rows, cols = dims(product, *size)
    torch.manual_seed(sum(size))
    across, m, k = size
    blocks = -(-k // 128)
    w, grid, wv = weight(rows, cols)
    work = bfz.linear_workspace(n, w)
    x = torch.randn(n, cols, device="cuda") * torch.exp(torch.randn(n, 1, device="cuda"))
    dy = torch.randn(n, rows, device="cuda") * torch.exp(torch.randn(n, 1, device="cuda")) * 1e-2
    (xc, xs), (dc, ds) = quantized(x, True), quantized(dy, True)
    xv, dv = value(xc, xs, True), value(dc, ds, True)
    for dtype in (F32, BF16, F16):
        _say("form", product, size, dtype, form(product, n, rows, cols, dtype))
        work.fill_(0xFF)
        buf, out = inside(across, m, dtype)
        if product == 0:
            bfz.linear(xc, w, grid, out, work, scales=xs, tiles=True)
            check(out.contiguous(), xv, wv.t(), blocks)
        elif product == 1:
            bfz.linear_grad_input(dc, w, grid, out, work, scales=ds, tiles=True)
            check(out.contiguous(), dv, wv, blocks)
        else:
            bfz.linear_grad_weight(dc, ds, xc, xs, out, work)
            check(out.contiguous(), dv.t(), xv, blocks)
        assert untouched(buf, across, m)
        # added to what is there, 16-byte aligned rows and others
        if product and dtype != F16:
            base = (torch.randn(across, m, device="cuda") * 1e-2).to(dtype)
            out = base.clone()
            if product == 1:
                bfz.linear_grad_input(dc, w, grid, out, work, scales=ds, tiles=True, accumulate=True)
                check(out, dv, wv, blocks, base)
            else:
                bfz.linear_grad_weight(dc, ds, xc, xs, out, work, accumulate=True)
                check(out, dv.t(), xv, blocks, base)


@pytest.mark.gpu
@pytest.mark.parametrize("size", FEW)
def test_few_tokens(size):
    n, rows, cols = size
    torch.manual_seed(sum(size))
    w, grid, wv = weight(rows, cols)
    x = torch.randn(n, cols, device="cuda")
    for tiles in (False, True):
        codes, scales = quantized(x, tiles)
        work = bfz.linear_workspace(n, w)
        for dtype in (F32, BF16, F16):
            _say("few", size, tiles, dtype, form(0, n, rows, cols, dtype))
            buf, out = inside(n, rows, dtype)
            bfz.linear(codes, w, grid, out, work, scales=scales, tiles=tiles)
            check(out.contiguous(), value(codes, scales, tiles), wv.t(), -(-cols // 128))
            assert untouched(buf, n, rows)
