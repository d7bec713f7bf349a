"""The vocabulary loss at the tile widths that training sizes take, checked
against 64 bits over several scale blocks.  Each case names the widths that it
is there for and asserts that the calls choose them.  Tolerances as in
test_gpu_vocab_loss.py."""
import ctypes as C
import math

import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_gpu_vocab_loss import _case, _check, _run, _say, _value

pytestmark = pytest.mark.gpu


def _shape(n, V, d, dw_type):
    out = (C.c_int64 * 7)()
    assert bfz.lib().bfz_vocab_loss_shape(n, V, d, 0 if dw_type == torch.float32 else 1, out) == 0
    return dict(zip(("loss_full", "loss", "piece", "grad_full", "grad", "hidden", "splits"), out))


CASES = [
    # whole rounds 256 wide, the rest 64 wide
    ((1013, 50001, 1000), dict(loss_full=49152, loss=64, grad_full=49152, grad=64, hidden=256, splits=16)),
    ((1499, 30011, 901), dict(loss=256, grad=256, hidden=256, splits=10)),
    ((400, 30001, 900), dict(loss_full=0, loss=256, grad=256, hidden=128, splits=16)),
    ((512, 16384, 2048), dict(loss=128, grad=128, hidden=128, splits=8)),
    ((260, 40000, 712), dict(loss=128, grad=128, hidden=64, splits=32)),
]


@pytest.mark.parametrize("dw_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("sizes,widths", CASES)
def test_wide_tiles(sizes, widths, kind, dw_type):
    _say("wide", sizes, kind, dw_type)
    n, V, d = sizes
    shape = _shape(n, V, d, dw_type)
    assert {k: shape[k] for k in widths} == widths
    h, w, grid, value, t = _case(n, V, d, kind)
    dloss = torch.rand(n, device="cuda") + 0.1
    _check(h, value, t, _run(h, w, grid, t, dloss, dw_type), dloss)


@pytest.mark.parametrize("sizes,widths", CASES[1:4])
def test_scattered_scales_in_wide_tiles(sizes, widths):
    """Tile scales from 2^-70 to 1, in no order, all-zero tiles of scale 1 among
    them."""
    _say("scattered scales", sizes)
    n, V, d = sizes
    h, codes, grid, _, t = _case(n, V, d, "fp8")
    fall = torch.randint(-70, 1, grid.shape, device="cuda")
    zero = torch.rand(grid.shape, device="cuda") < 0.1
    grid = torch.where(zero, 1.0, torch.ldexp(grid, fall)).contiguous()
    codes[zero.repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :d]] = 0
    dloss = torch.rand(n, device="cuda") + 0.1
    _check(h, _value(codes, grid), t, _run(h, codes, grid, t, dloss), dloss)


@pytest.mark.parametrize("dw_type", [torch.bfloat16, torch.float32])
def test_rows_past_32_bits(dw_type):
    """Gradient rows at offsets past 2^31 and 2^32 elements, each within its own
    roundings: dz, and the row's (2^-8 each in bf16).  In float32: the logits are
    exact here, lse's sum has 32 + V/2048 + 16 steps of 2^-24, p's argument 84,
    dz 2^-16 -- under 2^-14 together."""
    V, d, n = 1_060_000, 4096, 2
    _say("rows past 32 bits", dw_type)
    codes = torch.zeros(V, d, dtype=torch.uint8, device="cuda")
    codes[V - 1].fill_(0x38)  # 1.0
    codes[5].fill_(0x30)      # 0.5
    grid = torch.full((-(-V // 128), d // 128), 1.0, device="cuda")
    grid[-1], grid[0] = 1.0 / 512, 1.0 / 256
    h = torch.ones(n, d, device="cuda").to(torch.bfloat16)
    t = torch.tensor([V - 1, 5], device="cuda")
    _, lse, _, dw = _run(h, codes, grid, t, torch.ones(n, device="cuda"), dw_type)
    want = math.log(2 * math.e ** 8 + V - 2)  # z: 8 at both rows, 0 at the other V - 2
    for row in (6, 524_289, 600_000, 1_048_577, V - 2):
        expect = 2 * math.exp(-want)
        off = float((dw[row].double() - expect).abs().max()) / expect
        assert off <= (2.0 ** -14 if dw_type == torch.float32 else 2.05 * 2.0 ** -8), (row, off, dw[row, :3], expect)
    del dw
    torch.cuda.empty_cache()
