"""All three results of a norm that never clips."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_norm import _check, _norm, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [None, math.inf])
@pytest.mark.parametrize("count", [1, 7, 97])
def test_no_limit(count, limit):
    rng = np.random.default_rng(count)
    types = [torch.float32, torch.bfloat16, torch.float16]
    grads = [(torch.randn(int(rng.integers(1, 6000)), device="cuda") * 100).to(types[k % 3]) for k in range(count)]
    got = _norm(grads + [torch.empty(0, device="cuda")], limit)
    _check(got, _want(grads, math.inf))
    assert got[1] == 1.0
