"""Results that are made of exact products: float16 ones of every size, as float32
ones, any of up to 16 tokens, where the weight's bytes decide the time, and bfloat16
ones whose caller asks for them.

The operands are such that nothing but the last rounding may be off.  In every 8
columns of the sum two products are 2^15 and -2^15, all others multiples of 1/64
between -1 and 1, and the scales are 1: with up to four such pairs on the way at a
time and 4096 columns, every partial sum, whatever its order, is a multiple of 1/64
below 2^18, which binary32 holds.  An alignment of several products to the largest
of them, with 13 bits kept below it, loses all the small ones."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_linear import BF16, E4M3, F16, F32, _say

pytestmark = pytest.mark.gpu


def operands(m, n, k):
    """Codes (m, k) and (n, k), and the float64 product of their values."""
    gen = torch.Generator().manual_seed(m + n + k)
    a, b = (torch.randint(-8, 9, (z, k), generator=gen) / 8.0 for z in (m, n))
    for at in range(0, k - 7, 8):
        i, j = torch.randperm(8, generator=gen)[:2].tolist()
        a[:, at + i] = a[:, at + j] = 128.0
        b[:, at + i], b[:, at + j] = 256.0, -256.0
    want = (a.double().cuda() @ b.double().t().cuda())
    return codes(a), codes(b), want


def codes(x):
    """E4M3 codes of a matrix whose values E4M3 holds, rows on 16-byte
    boundaries."""
    c, _ = bfz.quantize_buffers(*x.shape)
    c.copy_(x.to(E4M3).view(torch.uint8))
    return c


def ones(*shape):
    return torch.ones(shape, device="cuda")


def blocks(n):
    return -(-n // 128)


FEW = [(1, 300, 640), (1, 4200, 1024), (5, 8300, 256), (16, 12400, 384), (20, 12400, 200), (33, 300, 4096), (48, 8200, 512), (64, 12400, 512)]


@pytest.mark.parametrize("n,rows,cols,dtype", [(*f, t) for f in FEW for t in (F32, BF16, F16) if t != BF16 or f[0] <= 16])
def test_few_tokens(n, rows, cols, dtype):
    x, w, want = operands(n, rows, cols)
    out = torch.full((n, rows), float("nan"), dtype=dtype, device="cuda")
    _say("exact, few", n, rows, cols, dtype)
    bfz.linear(x, w, ones(blocks(rows), blocks(cols)), out, bfz.linear_workspace(n, w), scales=ones(blocks(cols), n))
    assert torch.equal(out, want.float().to(dtype))


@pytest.mark.parametrize("n", [1, 4])
def test_few_values(n):
    """Values that the product quantizes itself: with a largest of 448 in each
    group of 128 their codes are the values."""
    rows, cols = 300, 512
    x, w, want = operands(n, rows, cols)
    values = x.contiguous().view(E4M3).float()
    for at in range(0, cols, 128):
        w[:, at:at + 8] = 0  # a whole group of 8, both of its large products among them
        values[:, at] = 448.0
    want = values.double() @ w.contiguous().view(E4M3).to(torch.float64).t()
    out = torch.full((n, rows), float("nan"), dtype=BF16, device="cuda")
    bfz.linear(values, w, ones(blocks(rows), blocks(cols)), out, bfz.linear_workspace(n, w, F32))
    assert torch.equal(out, want.float().to(BF16))


@pytest.mark.parametrize("n,rows,cols", [(20, 300, 640), (64, 12400, 512)])
def test_few_tokens_when_asked(n, rows, cols):
    x, w, want = operands(n, rows, cols)
    out = torch.full((n, rows), float("nan"), dtype=BF16, device="cuda")
    bfz.linear(x, w, ones(blocks(rows), blocks(cols)), out, bfz.linear_workspace(n, w), scales=ones(blocks(cols), n), exact=True)
    assert torch.equal(out, want.float().to(BF16))


@pytest.mark.parametrize("n,rows,cols", [(65, 300, 1001), (300, 513, 640), (1030, 1300, 912), (3590, 1700, 3600)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_all_products(n, rows, cols, dtype):
    """bfloat16 results with `exact`, which changes nothing for others."""
    _say("exact", n, rows, cols, dtype)
    exact = dtype == BF16
    x, w, want = operands(n, rows, cols)
    work = bfz.linear_workspace(n, w)
    grid = ones(blocks(rows), blocks(cols))
    out, dx, dw = (torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in ((n, rows), (n, cols), (rows, cols)))
    bfz.linear(x, w, grid, out, work, scales=ones(blocks(n), blocks(cols)), tiles=True, exact=exact)
    assert torch.equal(out, want.float().to(dtype))
    # contracted over rows: both operands' codes come as their transposes
    d, wt, want = operands(n, cols, rows)
    bfz.linear_grad_input(d, wt.t().contiguous(), grid, dx, work, scales=ones(blocks(n), blocks(rows)), tiles=True, exact=exact)
    assert torch.equal(dx, want.float().to(dtype))
    dt, xt, want = operands(rows, cols, n)
    d, _ = bfz.quantize_buffers(n, rows)
    x, _ = bfz.quantize_buffers(n, cols)
    d.copy_(dt.t())
    x.copy_(xt.t())
    bfz.linear_grad_weight(d, ones(blocks(n), blocks(rows)), x, ones(blocks(n), blocks(cols)), dw, work, exact=exact)
    assert torch.equal(dw, want.float().to(dtype))
