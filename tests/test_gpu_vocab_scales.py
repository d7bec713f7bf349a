"""Tile scales of an E4M3 head that fall or jump by more than binary32 could
carry in one unit: along the width (loss, lse) and along the vocabulary (dh),
at 16 tokens, which scale block by block, and above, where the sums are kept
in units of a tile scale.  Tolerances as in test_gpu_vocab_loss.py."""
import pytest
import torch

from tests.test_gpu_vocab_loss import _check, _run, _say, _value

pytestmark = pytest.mark.gpu

LADDERS = [(0, -59, -118), (0, -55, -110, -140), (0, -40, -80, -120), (-118, -59, 0), (0, -149, 0, -149), (60, 0, -60, 60), (-30, -90, -60, -149)]


def _case(n, V, d, seed):
    torch.manual_seed(seed)
    h = torch.randn(n, d, device="cuda").to(torch.bfloat16)
    codes = (torch.randn(V, d, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    t = torch.randint(0, V, (n,), device="cuda")
    if n > 4:
        t[1], t[3] = -100, V
    return h, codes, t


def _both(h, codes, grid, t, dw_type=torch.bfloat16):
    dloss = torch.rand(len(h), device="cuda") + 0.1
    _check(h, _value(codes, grid), t, _run(h, codes, grid, t, dloss, dw_type), dloss)


@pytest.mark.parametrize("n", [16, 17, 130, 300])
@pytest.mark.parametrize("exponents", LADDERS)
def test_ladders_along_the_width(n, exponents):
    _say("along the width", n, exponents)
    V, d = 400, 128 * len(exponents) - 32
    h, codes, t = _case(n, V, d, n)
    top = max(exponents)
    grid = torch.tensor([2.0 ** (e - top) if e > -149 else 2.0 ** -149 for e in exponents], device="cuda").repeat(-(-V // 128), 1)
    grid = (grid * 0.01).clamp(min=2.0 ** -149).contiguous()
    _both(h, codes, grid, t)


@pytest.mark.parametrize("n", [16, 17, 300, 9000])  # 9000: one sum over all rows
@pytest.mark.parametrize("exponents", LADDERS)
def test_ladders_along_the_vocabulary(n, exponents):
    _say("along the vocabulary", n, exponents)
    V, d = 128 * len(exponents) - 40, 272
    h, codes, t = _case(n, V, d, n + 1)
    top = max(exponents)
    grid = torch.tensor([2.0 ** (e - top) if e > -149 else 2.0 ** -149 for e in exponents], device="cuda")[:, None].repeat(1, -(-d // 128))
    grid = (grid * 0.01).clamp(min=2.0 ** -149).contiguous()
    _both(h, codes, grid, t)


@pytest.mark.parametrize("n", [16, 17, 300])
@pytest.mark.parametrize("low", [-62, -90])
def test_a_zero_tile_bounds_nothing(n, low):
    """An all-zero tile has scale 1 by the step's rule: what follows it, however
    small, is the whole result.  The small logits are all of dh."""
    _say("zero tile", n, low)
    V, d = 600, 300
    h, codes, t = _case(n, V, d, n + 2)
    for axis in (0, 1):
        c, grid = codes.clone(), torch.full((-(-V // 128), -(-d // 128)), 2.0 ** low, device="cuda")
        c.view(V, d).narrow(axis, 0, 128).zero_()
        grid.narrow(axis, 0, 1).fill_(1.0)
        _both(h, c, grid, t)


@pytest.mark.parametrize("n", [16, 17, 300])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_a_nan_scale_is_seen(n, at):
    V, d = 300, 512
    h, codes, t = _case(n, V, d, n + 3)
    grid = torch.full((-(-V // 128), -(-d // 128)), 0.001, device="cuda")
    grid[1, at] = float("nan")
    loss, lse = _run(h, codes, grid, t)
    assert bool(torch.isnan(lse).all())


@pytest.mark.parametrize("n", [16, 17, 300])
@pytest.mark.parametrize("share", [0.5, 1.0])
def test_zero_scales(n, share):
    """A grid that nothing has been written to yet."""
    V, d = 700, 900
    h, codes, t = _case(n, V, d, n + 4)
    grid = torch.full((-(-V // 128), -(-d // 128)), 0.001, device="cuda")
    grid[torch.rand(grid.shape, device="cuda") < share] = 0.0
    _both(h, codes, grid, t)
