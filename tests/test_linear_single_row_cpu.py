"""One row of codes out of rows that do not start on 16-byte boundaries: its stride
says nothing (CPU: the library's call is a stand-in that keeps its arguments)."""
import sys

import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_layer_refusals_cpu import _z, at_home  # noqa: F401


def test_single_row(at_home, monkeypatch):  # noqa: F811
    args = {}

    class Library:
        def bfz_quantize(self, *a):
            args["quantize"] = a
            return 0

        def bfz_linear(self, *a):
            args["linear"] = a
            return 0

    linear = sys.modules["blockwise_fp8_zero_amd.linear"]
    monkeypatch.setattr(linear, "lib", Library)
    monkeypatch.setattr(linear, "raw_stream", lambda *a: 0)
    monkeypatch.setattr(linear, "_work_bytes", lambda *sizes: 256)
    codes = _z(1, 130, dtype=torch.uint8)[:, :100]
    assert codes.stride(0) == 130
    bfz.quantize(_z(1, 100), codes, _z(1, 1))
    assert args["quantize"][8] == 112
    bfz.linear(codes, _z(40, 100, dtype=torch.uint8), _z(1, 1), _z(1, 40), _z(256, dtype=torch.uint8), scales=_z(1, 1))
    assert args["linear"][2] == 112
