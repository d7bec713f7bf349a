"""A row of E4M3 codes is its value, code * tile scale in binary32, times `scale`:
bit for bit, also where scale times the tile's own would leave binary32."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,d,ld", [(300, 256, 256), (300, 200, 208), (257, 131, 131), (130, 4, 4), (400, 1000, 1000)])
@pytest.mark.parametrize("scale", [1.0, 0.03125, 31.6227766, 2.0 ** 100, 2.0 ** -60])
def test_value_then_scale(V, d, ld, out_type, scale):
    torch.manual_seed(V + d)
    table = torch.randint(0, 256, (V, ld), dtype=torch.uint8, device="cuda")
    table[(table & 0x7F) == 0x7F] = 0x7E  # no NaN
    table = table[:, :d]
    exponents = torch.tensor([-149, -140, -126, -80, -20, 0, 20, 90], device="cuda")
    cells = (-(-V // 128), -(-d // 128))
    grid = torch.ldexp(torch.ones(cells, device="cuda"), exponents[torch.randint(0, 8, cells, device="cuda")])
    grid = torch.where(grid > 2.0 ** -126, grid * 1.37, grid).contiguous()
    ids = torch.randint(-2, V + 2, (700,), device="cuda")
    out = torch.full((700, d), float("nan"), device="cuda").to(out_type)
    bfz.embed(ids, table, out, scale=scale, grid=grid)
    up = grid.repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :d]
    value = table.contiguous().view(torch.float8_e4m3fn).float() * up
    there = (ids >= 0) & (ids < V)
    want = torch.where(there[:, None], value[ids.clamp(0, V - 1)] * scale, 0.0).to(out_type)
    assert torch.equal(out.isinf(), want.isinf()) and torch.equal(out, want)
