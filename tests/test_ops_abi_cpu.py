"""The operators around the step refuse bad arguments before any launch (CPU:
pointers here are never followed)."""
import ctypes as C

import pytest
import torch

import blockwise_fp8_zero_amd as bfz


class _Tensor(C.Structure):
    _fields_ = [("data", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32), ("reserved", C.c_int32)]


P = C.c_void_p
A, B, W = P(0x10000), P(0x20000), P(0x30000)
EINVAL, EALIGN, ESTATE = bfz.BFZ_EINVAL, bfz.BFZ_EALIGN, bfz.BFZ_ESTATE


def _list(*items):
    arr = (_Tensor * max(1, len(items)))()
    for k, it in enumerate(items):
        arr[k] = _Tensor(*it)
    return C.cast(arr, P)


def test_grad_norm_refusals():
    f = bfz.lib().bfz_grad_norm
    one = _list((0x1000, 5, 0, 0))
    assert f(None, 1, 1.0, None, A, B, W, None) == EINVAL
    assert f(one, -1, 1.0, None, A, B, W, None) == EINVAL
    for bad in (0.0, -1.0, float("nan")):
        assert f(one, 1, bad, None, A, B, W, None) == EINVAL
    assert f(one, 1, 1.0, None, A, B, None, None) == EINVAL
    assert f(one, 1, 1.0, None, A, B, P(0x30008), None) == EALIGN
    assert f(one, 1, 1.0, P(0x10004), A, B, W, None) == EALIGN
    assert f(one, 1, 1.0, None, P(0x10002), B, W, None) == EALIGN
    assert f(one, 1, 1.0, None, A, P(0x10001), W, None) == EALIGN
    for t, rc in (((0, 5, 0, 0), EINVAL), ((0x1000, -1, 0, 0), EINVAL), ((0x1000, 5, 3, 0), EINVAL), ((0x1000, 5, 9, 0), EINVAL),
                  ((0x1000, 5, 0, 1), EINVAL), ((0x1002, 5, 0, 0), EALIGN), ((0x1001, 5, 1, 0), EALIGN)):
        assert f(_list(t), 1, 1.0, None, A, B, W, None) == rc, t
    assert "gradient 0" in bfz.lib().bfz_last_error().decode()


def test_shard_norm_and_coef_refusals():
    L = bfz.lib()
    plan = bfz.Plan([(1, 200, 200)])
    g = C.cast((P * 1)(0x1000), P)
    assert L.bfz_shard_grad_norm(None, g, 1.0, None, A, B, W, None) == EINVAL
    assert L.bfz_shard_grad_norm(plan.handle, None, 1.0, None, A, B, W, None) == EINVAL
    assert L.bfz_shard_grad_norm(plan.handle, g, 0.0, None, A, B, W, None) == EINVAL
    assert L.bfz_shard_grad_norm(plan.handle, g, 1.0, None, A, B, None, None) == EINVAL
    assert L.bfz_shard_grad_norm(plan.handle, g, 1.0, None, A, B, W, None) == ESTATE  # no device here
    assert L.bfz_clip_coef(None, 1.0, A, B, None) == EINVAL
    assert L.bfz_clip_coef(P(0x1004), 1.0, A, B, None) == EALIGN
    assert L.bfz_clip_coef(A, -1.0, A, B, None) == EINVAL
    plan.close()


def test_clip_refusals():
    f = bfz.lib().bfz_clip_grads
    g = _list((0x1000, 5, 0, 0))
    assert f(g, g, 1, None, None) == EINVAL
    assert f(g, g, 1, P(0x1002), None) == EALIGN
    assert f(g, None, 1, A, None) == EINVAL
    assert f(g, _list((0x2000, 6, 0, 0)), 1, A, None) == EINVAL
    assert f(g, _list((0x1000, 5, 1, 0)), 1, A, None) == EINVAL
    assert f(g, _list((0x2000, 5, 3, 0)), 1, A, None) == EINVAL
    assert f(g, _list((0x2002, 5, 0, 0)), 1, A, None) == EALIGN


def test_clipped_step_refusals():
    L = bfz.lib()
    hp = bfz.AdamW(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    st = [P(0x10000 * k) for k in range(1, 7)]
    assert L.bfz_adamw_fp8_step_clip(*st, 1, C.byref(hp), None, None, None) == EINVAL
    assert L.bfz_adamw_fp8_step_clip(*st, 1, C.byref(hp), None, P(0x1002), None) == EALIGN
    assert L.bfz_adamw_fp8_step_clip(*st, -1, C.byref(hp), None, A, None) == EINVAL
    plan = bfz.Plan([(1, 200, 200)])
    g = C.cast((P * 1)(0x1000), P)
    assert L.bfz_fold_adamw_fp8_step_clip(plan.handle, g, *st[:5], C.byref(hp), None, None, None) == EINVAL
    assert L.bfz_fold_adamw_fp8_step_clip(plan.handle, g, *st[:5], C.byref(hp), None, A, None) == ESTATE
    assert L.bfz_fold_adamw_fp8_step_unpack_clip(plan.handle, g, *st[:5], g, g, C.byref(hp), None, None, None) == EINVAL
    assert L.bfz_fold_adamw_fp8_step_unpack_t_clip(plan.handle, g, *st[:5], g, g, g, g, C.byref(hp), None, None, None) == EINVAL
    plan.close()


def _embed(ids=A, wide=1, n=4, table=B, tt=0, grid=None, V=10, d=8, tld=8, out=W, ot=0, old=8):
    return bfz.lib().bfz_embed(ids, wide, n, table, tt, grid, V, d, tld, 1.0, out, ot, old, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(ids=None), EINVAL), (dict(n=-1), EINVAL), (dict(V=0), EINVAL), (dict(d=0), EINVAL), (dict(V=1 << 28), EINVAL),
    (dict(n=1 << 28), EINVAL), (dict(table=None), EINVAL), (dict(out=None), EINVAL), (dict(tt=4), EINVAL), (dict(ot=3), EINVAL),
    (dict(tt=3), EINVAL), (dict(grid=A), EINVAL), (dict(tt=3, grid=P(0x1001)), EALIGN), (dict(tld=7), EINVAL), (dict(old=7), EINVAL),
    (dict(ids=P(0x1004)), EALIGN), (dict(ids=P(0x1002), wide=0), EALIGN), (dict(table=P(0x1002)), EALIGN), (dict(out=P(0x1001), ot=1), EALIGN),
])
def test_embed_refusals(kw, rc):
    assert _embed(**kw) == rc
    assert "bfz_embed" in bfz.lib().bfz_last_error().decode()


def _embed_grad(ids=A, wide=1, n=4, dout=B, it=0, dld=8, V=10, d=8, dt=P(0x50000), ot=0, tld=8, work=W):
    return bfz.lib().bfz_embed_grad(ids, wide, n, dout, it, dld, V, d, 1.0, 0, dt, ot, tld, work, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(ids=None), EINVAL), (dict(n=-1), EINVAL), (dict(V=0), EINVAL), (dict(d=0), EINVAL), (dict(dout=None), EINVAL),
    (dict(dt=None), EINVAL), (dict(it=3), EINVAL), (dict(ot=3), EINVAL), (dict(dld=7), EINVAL), (dict(tld=1), EINVAL),
    (dict(work=None), EINVAL), (dict(work=P(0x30008)), EALIGN), (dict(dout=P(0x1002)), EALIGN), (dict(dt=P(0x1001), ot=2), EALIGN),
    (dict(n=1 << 27, d=4096, dld=4096, tld=4096), EINVAL),
])
def test_embed_grad_refusals(kw, rc):
    assert _embed_grad(**kw) == rc


def test_work_sizes():
    L = bfz.lib()
    assert L.bfz_norm_work_bytes() > 64
    assert L.bfz_embed_grad_work_bytes(-1, 8) == 0 and L.bfz_embed_grad_work_bytes(8, 0) == 0
    sizes = [L.bfz_embed_grad_work_bytes(n, 100) for n in (0, 1, 100, 16383, 16384, 20000, 70000)]
    assert sizes == sorted(sizes)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        bfz.grad_norm([x], None, x)
    with pytest.raises(TypeError):
        bfz.embed(torch.zeros(4, dtype=torch.long), x, x)
    with pytest.raises(TypeError):
        bfz.embed_grad(torch.zeros(4, dtype=torch.long), x, x, x)


def _loss(grad=False, hidden=A, hld=8, n=4, weight=B, wt=1, wld=8, grid=None, V=10, d=8, t=P(0x40000), wide=1, loss=P(0x50000),
          lse=P(0x60000), work=W, dloss=P(0x70000), dh=P(0x80000), dhld=8, dw=P(0x90000), dwt=1, dwld=8):
    L = bfz.lib()
    if not grad:
        return L.bfz_vocab_loss(hidden, hld, n, weight, wt, wld, grid, V, d, t, wide, loss, lse, work, None)
    return L.bfz_vocab_loss_grad(hidden, hld, n, weight, wt, wld, grid, V, d, t, wide, lse, dloss, dh, dhld, dw, dwt, dwld, 0, work,
                                 None)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(hidden=None), EINVAL), (dict(weight=None), EINVAL), (dict(t=None), EINVAL), (dict(lse=None), EINVAL), (dict(work=None), EINVAL),
    (dict(n=-1), EINVAL), (dict(V=0), EINVAL), (dict(d=0), EINVAL), (dict(n=1 << 25), EINVAL), (dict(V=1 << 28), EINVAL),
    (dict(d=1 << 21, hld=1 << 21, wld=1 << 21), EINVAL), (dict(n=1 << 24, V=1 << 27), EINVAL), (dict(n=1 << 24, d=1 << 20, hld=1 << 20, wld=1 << 20), EINVAL), (dict(wt=0), EINVAL), (dict(wt=3), EINVAL),
    (dict(grid=A), EINVAL), (dict(wt=3, grid=P(0x1002)), EALIGN), (dict(hld=7), EINVAL), (dict(wld=7), EINVAL), (dict(wld=1 << 22), EINVAL),
    (dict(hidden=P(0x1001)), EALIGN), (dict(weight=P(0x1001)), EALIGN), (dict(t=P(0x1004)), EALIGN), (dict(t=P(0x1002), wide=0), EALIGN),
    (dict(lse=P(0x1002)), EALIGN), (dict(work=P(0x1010)), EALIGN),
])
def test_vocab_loss_refusals(grad, kw, rc):
    assert _loss(grad, **kw) == rc
    assert "bfz_vocab_loss" in bfz.lib().bfz_last_error().decode()


@pytest.mark.parametrize("kw,rc", [
    (dict(dloss=None), EINVAL), (dict(dloss=P(0x1002)), EALIGN), (dict(dh=P(0x1001)), EALIGN), (dict(dhld=7), EINVAL),
    (dict(dwt=2), EINVAL), (dict(dwt=3), EINVAL), (dict(dwld=7), EINVAL), (dict(dw=P(0x1002), dwt=0), EALIGN),
])
def test_vocab_loss_grad_refusals(kw, rc):
    assert _loss(True, **kw) == rc


def test_vocab_loss_refuses_a_null_loss():
    assert _loss(loss=None) == EINVAL and _loss(loss=P(0x1001)) == EALIGN


def test_vocab_loss_work_sizes():
    f = bfz.lib().bfz_vocab_loss_work_bytes
    assert f(-1, 10, 8, 1, 0) == 0 and f(4, 0, 8, 1, 0) == 0 and f(4, 10, 8, 0, 0) == 0
    assert 0 < f(4, 10, 8, 1, 0) <= f(4, 10, 8, 1, 1)
    # a workspace for n tokens serves every smaller batch
    for V, d, t in ((131072, 4096, 3), (50001, 1000, 1), (300, 64, 3), (1 << 20, 512, 1)):
        for grad in (0, 1):
            sizes = [f(n, V, d, t, grad) for n in (0, 1, 16, 17, 100, 1000, 3000, 4000, 8192, 16384, 16385, 40000)]
            assert sizes == sorted(sizes), (V, d, t, grad, sizes)
    # dz and the padded copy are bounded, whatever the vocabulary
    assert f(8192, 1 << 20, 4096, 3, 1) < 4 << 30
