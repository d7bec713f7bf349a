"""Workspaces of types that no call takes are refused as the calls refuse them."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz


def test_linear_workspace():
    weight = torch.zeros(40, 32, dtype=torch.uint8)
    for dtype in (torch.float64, torch.int32, float):
        with pytest.raises(TypeError, match="x_dtype"):
            bfz.linear_workspace(5, weight, dtype)
    codes = bfz.linear_workspace(5, weight).numel()
    assert codes == bfz.linear_workspace(5, weight, torch.uint8).numel() == bfz.linear_workspace(5, weight, torch.float8_e4m3fn).numel()
    assert codes < bfz.linear_workspace(5, weight, torch.bfloat16).numel()
