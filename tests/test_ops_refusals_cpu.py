"""More refusals of the operators around the step (CPU: nothing is launched)."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_ops_abi_cpu import EALIGN, EINVAL, P, _embed, _embed_grad, _loss


def test_rounded_float_dweight():
    assert _loss(True, dw=P(0x1002), dwt=4) == EALIGN and _loss(True, dwt=4, dwld=7) == EINVAL
    assert _loss(True, dwt=5) == EINVAL and _loss(True, wt=4) == EINVAL
    assert _embed(ot=4) == EINVAL and _embed_grad(it=4) == EINVAL and _embed_grad(ot=4) == EINVAL
