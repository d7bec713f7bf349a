"""Two steps of one AdamWList at a time, each with the gradients that it was given
(CPU: the library's call is a stand-in that reads the table)."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from blockwise_fp8_zero_amd import adamw_list
from tests.test_layer_refusals_cpu import _z, at_home  # noqa: F401

HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)


@pytest.mark.parametrize("of_list", [False, True])
def test_a_step_within_a_step(at_home, monkeypatch, of_list):  # noqa: F811
    """The second begins while the first one's call runs, as another thread's may:
    ctypes lets go of the interpreter there."""
    def some(dtype):
        return [_z(300, dtype=dtype), _z(30, dtype=dtype)]

    p, own, first, second = some(torch.float32), some(torch.float32), some(torch.bfloat16), some(torch.float16)
    opt = bfz.AdamWList(p, some(torch.float32), some(torch.float32), grads=own)
    seen = []

    class Library:
        def bfz_adamw_list(self, words, *rest):
            if not seen:
                seen.append(None)
                opt.step(HP) if of_list else opt.step(HP, grads=second)
                seen[0] = table(words)
            else:
                seen.append(table(words))
            return 0

    def table(words):
        return [(words[9 * k + 1], words[9 * k + 7] >> 32) for k in range(len(p))]

    def of(grads, code):
        return [(g.data_ptr(), code) for g in grads]

    monkeypatch.setattr(adamw_list, "lib", Library)
    monkeypatch.setattr(adamw_list, "raw_stream", lambda *a: 0)
    opt.step(HP, grads=first)
    assert seen[0] == of(first, 1)
    assert seen[1] == (of(own, 0) if of_list else of(second, 2))
    seen[:] = [None]
    opt.step(HP)
    assert seen[1] == of(own, 0)
