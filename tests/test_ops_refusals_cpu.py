"""More refusals of the operators around the step (CPU: nothing is launched)."""
import pytest
import torch

import blockwise_fp8_zero_amd as bfz
from tests.test_ops_abi_cpu import EALIGN, EINVAL, P, _embed, _embed_grad, _loss


def test_rounded_float_dweight():
    assert _loss(True, dw=P(0x1002), dwt=4) == EALIGN and _loss(True, dwt=4, dwld=7) == EINVAL
    assert _loss(True, dwt=5) == EINVAL and _loss(True, wt=4) == EINVAL
    assert _embed(ot=4) == EINVAL and _embed_grad(it=4) == EINVAL and _embed_grad(ot=4) == EINVAL


class _Elsewhere(torch.Tensor):
    """Stands for a tensor of cuda:1."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


class _Here(_Elsewhere):
    def get_device(self):
        return 0


def _calls():
    """(name of the tensor put elsewhere, the call): every tensor of every call in
    turn.  The refusal comes before any launch, and a call whose tensors are all
    at home is not made."""
    def z(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype).as_subclass(_Here)

    b16 = torch.bfloat16
    plan = bfz.Plan([(1, 8, 16)])
    work = dict(work=z(1 << 20, dtype=torch.uint8))
    one = dict(norm=z(1), coef=z(1), sumsq=z(1, dtype=torch.float64))
    loss = dict(hidden=z(4, 16, dtype=b16), weight=z(8, 16, dtype=torch.uint8), targets=z(4, dtype=torch.int64), lse=z(4), grid=z(1, 1),
                **work)
    forms = [
        (bfz.grad_norm, dict(grads=[z(5)], **one, **work)),
        (lambda **k: bfz.shard_grad_norm(plan, **k), dict(grads=[z(1, 8, 16)], **one, **work)),
        (lambda **k: bfz.clip_coef(max_norm=1.0, **k), one),
        (bfz.clip_grads, dict(grads=[z(5)], coef=z(1), outs=[z(5)])),
        (bfz.embed, dict(ids=z(4, dtype=torch.int64), table=z(8, 16, dtype=torch.uint8), out=z(4, 16), grid=z(1, 1))),
        (bfz.embed_grad, dict(ids=z(4, dtype=torch.int64), dout=z(4, 16), dtable=z(8, 16), **work)),
        (bfz.vocab_loss, dict(loss=z(4), **loss)),
        (bfz.vocab_loss_grad, dict(dloss=z(4), dhidden=z(4, 16, dtype=b16), dweight=z(8, 16), **loss)),
    ]
    for f, kw in forms:
        for name, t in kw.items():
            moved = [x.as_subclass(_Elsewhere) for x in t] if isinstance(t, list) else t.as_subclass(_Elsewhere)
            yield name, f, {**kw, name: moved}


def test_tensors_of_another_device(monkeypatch):
    from blockwise_fp8_zero_amd import _tensors
    _tensors._load()
    monkeypatch.setattr(_tensors, "_current", lambda: 0)
    monkeypatch.setattr(_tensors, "raw_stream", lambda stream, home: pytest.fail("nothing may be launched"))
    for module in (bfz.norm, bfz.embedding, bfz.vocab_loss.__globals__):
        names = module if isinstance(module, dict) else vars(module)
        monkeypatch.setitem(names, "raw_stream", _tensors.raw_stream)
    count = 0
    for name, f, kw in _calls():
        with pytest.raises(ValueError, match="current device is cuda:0"):
            f(**kw)
        count += 1
    assert count == 40


def test_factor_and_stream_of_another_device(monkeypatch):
    from blockwise_fp8_zero_amd import _tensors
    _tensors._load()
    monkeypatch.setattr(_tensors, "_current", lambda: 0)
    with pytest.raises(ValueError, match="grad_scale"):
        bfz._clip("fold_adamw_fp8_step", torch.zeros(1).as_subclass(_Elsewhere))

    class Stream:
        device_index, cuda_stream = 1, 0x1000

    with pytest.raises(ValueError, match="stream"):
        bfz.raw_stream(Stream())


def test_vocab_loss_shape():
    import ctypes as C
    f, out = bfz.lib().bfz_vocab_loss_shape, (C.c_int64 * 7)()
    assert f(100, 1000, 64, 1, None) == EINVAL and f(0, 1000, 64, 1, out) == EINVAL and f(100, 1 << 28, 64, 1, out) == EINVAL
    for n, V, d in ((1, 300, 64), (16, 5000, 200), (17, 600, 136), (1013, 50001, 1000), (8192, 131072, 4096), (100000, 131072, 512)):
        for dw in (0, 1, 4):
            assert f(n, V, d, dw, out) == 0
            full, width, piece, grad_full, grad_width, hidden, splits = out
            assert 0 <= full < V and full % 256 == 0 and 0 <= grad_full < V and grad_full % 256 == 0 and piece % 256 == 0
            assert {width, grad_width} <= ({16} if n <= 16 else {256, 128, 64}) and hidden in (256, 128, 64)
            assert 1 <= splits <= 64 and splits * n <= max(16384, n)
            # a piece's dz stays within what the workspace has for it
            assert n * piece * (4 if dw == 0 else 2) <= max(1 << 29, n * 2048)
