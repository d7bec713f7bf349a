"""The quantizer, the linear products, layer norm and AdamW over many tensors refuse
bad arguments before any launch (CPU: pointers here are never followed)."""
import ctypes as C

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

P = C.c_void_p
EINVAL, EALIGN = bfz.BFZ_EINVAL, bfz.BFZ_EALIGN
X, S, W, G, O, WORK = (P(0x10000 * k) for k in range(1, 7))
F32, BF16, F16, E4M3 = 0, 1, 2, 3


def _quantize(x=X, xt=0, xld=40, n=5, d=40, tiles=0, codes=W, cld=48, scales=S, sld=5):
    return bfz.lib().bfz_quantize(x, xt, xld, n, d, tiles, 0, codes, cld, scales, sld, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(xt=3), EINVAL), (dict(xt=9), EINVAL), (dict(xld=39), EINVAL), (dict(n=-1), EINVAL), (dict(d=0), EINVAL),
    (dict(n=(1 << 24) + 1), EINVAL), (dict(d=(1 << 20) + 1, xld=1 << 21, cld=1 << 21), EINVAL), (dict(n=1 << 24, d=1 << 20, xld=1 << 20, cld=1 << 20, sld=1 << 24), EINVAL),
    (dict(codes=None), EINVAL), (dict(cld=39), EINVAL), (dict(cld=40), EALIGN), (dict(codes=P(0x1008)), EALIGN), (dict(cld=(1 << 21) + 16), EINVAL),
    (dict(scales=None), EINVAL), (dict(sld=4), EINVAL), (dict(tiles=1, sld=0), EINVAL), (dict(scales=P(0x1002)), EALIGN), (dict(x=P(0x1002)), EALIGN),
    (dict(x=P(0x1001), xt=1), EALIGN),
])
def test_quantize(kw, rc):
    assert _quantize(**kw) == rc
    assert "bfz_quantize" in bfz.lib().bfz_last_error().decode()


def _linear(x=X, xt=E4M3, xld=48, s=S, sld=5, tiles=0, n=5, w=W, wld=33, g=G, rows=300, cols=33, o=O, ot=0, old=300, work=WORK):
    return bfz.lib().bfz_linear(x, xt, xld, s, sld, tiles, n, w, wld, g, rows, cols, o, ot, old, work, None)


COMMON = [
    (dict(w=None), EINVAL), (dict(wld=32), EINVAL), (dict(wld=(1 << 21) + 1), EINVAL), (dict(g=None), EINVAL), (dict(g=P(0x1001)), EALIGN), (dict(n=-1), EINVAL),
    (dict(rows=0), EINVAL), (dict(cols=0), EINVAL), (dict(n=(1 << 24) + 1), EINVAL), (dict(o=None), EINVAL), (dict(ot=3), EINVAL), (dict(ot=4), EINVAL),
    (dict(o=P(0x1002)), EALIGN), (dict(o=P(0x1001), ot=1), EALIGN), (dict(work=None), EINVAL), (dict(work=P(0x1080)), EALIGN), (dict(s=None), EINVAL),
    (dict(s=P(0x1002)), EALIGN), (dict(sld=4), EINVAL), (dict(sld=(1 << 24) + 1), EINVAL),
]


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(x=None), EINVAL), (dict(xld=32), EINVAL), (dict(xld=40), EALIGN), (dict(x=P(0x1004)), EALIGN), (dict(old=299), EINVAL), (dict(xt=4), EINVAL),
    (dict(xt=1), EINVAL), (dict(xt=1, s=None, tiles=1), EINVAL), (dict(xt=1, s=None, xld=32), EINVAL), (dict(xt=0, s=None, x=P(0x1002)), EALIGN),
    (dict(tiles=1, sld=0), EINVAL), (dict(n=1 << 24, rows=1 << 20, old=1 << 20, sld=1 << 24), EINVAL),
])
def test_linear(kw, rc):
    assert _linear(**kw) == rc
    assert "bfz_linear" in bfz.lib().bfz_last_error().decode()


def _grad_input(x=X, xld=304, s=S, sld=5, tiles=0, n=5, w=W, wld=33, g=G, rows=300, cols=33, o=O, ot=0, old=33, work=WORK):
    return bfz.lib().bfz_linear_grad_input(x, xld, s, sld, tiles, n, w, wld, g, rows, cols, o, ot, old, 0, work, None)


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(x=None), EINVAL), (dict(xld=299), EINVAL), (dict(xld=300), EALIGN), (dict(old=32), EINVAL)])
def test_grad_input(kw, rc):
    assert _grad_input(**kw) == rc


def _grad_weight(x=X, xld=304, s=S, sld=3, y=W, yld=48, t=G, tld=1, n=5, rows=300, cols=33, o=O, ot=0, old=33, work=WORK):
    return bfz.lib().bfz_linear_grad_weight(x, xld, s, sld, y, yld, t, tld, n, rows, cols, o, ot, old, 0, work, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(s=None), EINVAL), (dict(t=None), EINVAL), (dict(sld=2), EINVAL), (dict(tld=0), EINVAL),
    (dict(xld=300), EALIGN), (dict(yld=40), EALIGN), (dict(yld=32), EINVAL), (dict(o=None), EINVAL), (dict(ot=3), EINVAL), (dict(old=32), EINVAL),
    (dict(n=-1), EINVAL), (dict(work=None), EINVAL), (dict(work=P(0x1010)), EALIGN), (dict(t=P(0x1001)), EALIGN),
    (dict(rows=1 << 20, cols=1 << 20, xld=1 << 20, yld=1 << 20, sld=1 << 13, tld=1 << 13, old=1 << 20), EINVAL),
])
def test_grad_weight(kw, rc):
    assert _grad_weight(**kw) == rc


def test_work_sizes():
    f = bfz.lib().bfz_linear_work_bytes
    assert f(-1, 10, 10, 3, 0) == 0 and f(1, 0, 10, 3, 0) == 0 and f(1, 10, 0, 3, 0) == 0 and f(1, 10, 10, 4, 0) == 0
    for dtype in (0, 1, 2, 3):
        for copy in (0, 1):
            sizes = [f(n, 1000, 1001, dtype, copy) for n in (0, 1, 5, 100, 4096, 100000)]
            assert sizes == sorted(sizes) and sizes[0] > 0
    assert f(8, 64, 64, 3, 0) <= f(8, 64, 64, 3, 1) <= f(8, 64, 64, 0, 1)
    g = bfz.lib().bfz_layer_norm_work_bytes
    assert g(-1, 10) == 0 and g(5, 0) == 0 and g(5, 32769) == 0
    for d in (1, 700, 1500, 4000, 8000, 16000, 32768):
        sizes = [g(n, d) for n in (0, 1, 5, 100, 4096, 100000)]
        assert sizes == sorted(sizes) and sizes[0] > 0


def _norm(x=X, xt=0, xld=40, n=5, d=40, w=W, b=G, pt=0, eps=1e-5, o=O, ot=0, old=40, mean=S, rstd=S):
    return bfz.lib().bfz_layer_norm(x, xt, xld, n, d, w, b, pt, eps, o, ot, old, mean, rstd, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(o=None), EINVAL), (dict(xt=3), EINVAL), (dict(ot=3), EINVAL), (dict(pt=3), EINVAL), (dict(xld=39), EINVAL), (dict(old=39), EINVAL),
    (dict(n=-1), EINVAL), (dict(d=0), EINVAL), (dict(d=32769, xld=40000, old=40000), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(w=P(0x1002)), EALIGN), (dict(b=P(0x1001), pt=1), EALIGN),
    (dict(mean=P(0x1002)), EALIGN), (dict(rstd=P(0x1001)), EALIGN), (dict(x=P(0x1002)), EALIGN),
])
def test_layer_norm(kw, rc):
    assert _norm(**kw) == rc
    assert "bfz_layer_norm" in bfz.lib().bfz_last_error().decode()


def _norm_grad(d_=X, dt=0, dld=40, x=X, xt=0, xld=40, n=5, d=40, w=W, pt=0, mean=S, rstd=S, o=O, ot=0, old=40, dw=G, db=G, gt=0, work=WORK):
    return bfz.lib().bfz_layer_norm_grad(d_, dt, dld, x, xt, xld, n, d, w, pt, mean, rstd, o, ot, old, dw, db, gt, 0, work, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(d_=None), EINVAL), (dict(x=None), EINVAL), (dict(dt=3), EINVAL), (dict(xt=3), EINVAL), (dict(pt=3), EINVAL), (dict(gt=3), EINVAL), (dict(ot=3), EINVAL),
    (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dld=39), EINVAL), (dict(xld=39), EINVAL), (dict(old=39), EINVAL), (dict(work=None), EINVAL),
    (dict(work=P(0x1010)), EALIGN), (dict(dw=P(0x1002)), EALIGN), (dict(db=P(0x1002)), EALIGN), (dict(mean=P(0x1002)), EALIGN), (dict(n=-1), EINVAL),
])
def test_layer_norm_grad(kw, rc):
    assert _norm_grad(**kw) == rc


class _Tensor(C.Structure):
    _fields_ = [("param", P), ("grad", P), ("m", P), ("v", P), ("m_scale", P), ("v_scale", P), ("n", C.c_int64),
                ("param_dtype", C.c_int32), ("grad_dtype", C.c_int32), ("state_dtype", C.c_int32), ("reserved", C.c_int32)]


def _adamw(hp=None, scale=None, count=1, **kw):
    t = dict(param=0x1000, grad=0x2000, m=0x3000, v=0x4000, m_scale=None, v_scale=None, n=5, param_dtype=0, grad_dtype=0, state_dtype=0, reserved=0)
    t.update(kw)
    h = bfz.AdamW(**{**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1), **(hp or {})})
    return bfz.lib().bfz_adamw_list(C.byref(_Tensor(**t)), count, C.byref(h), scale, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(param=None), EINVAL), (dict(grad=None), EINVAL), (dict(m=None), EINVAL), (dict(v=None), EINVAL), (dict(n=-1), EINVAL), (dict(reserved=1), EINVAL),
    (dict(param_dtype=3), EINVAL), (dict(grad_dtype=3), EINVAL), (dict(state_dtype=1), EINVAL), (dict(state_dtype=3), EINVAL), (dict(m_scale=0x5000), EINVAL),
    (dict(state_dtype=3, m_scale=0x5000), EINVAL), (dict(state_dtype=3, m_scale=0x5001, v_scale=0x6000), EALIGN), (dict(param=0x1002), EALIGN),
    (dict(grad=0x1001, grad_dtype=1), EALIGN), (dict(m=0x3002), EALIGN), (dict(scale=P(0x1002)), EALIGN), (dict(count=-1), EINVAL),
    (dict(hp=dict(eps=0.0)), EINVAL), (dict(hp=dict(beta1=1.0)), EINVAL), (dict(hp=dict(step=0)), EINVAL), (dict(hp=dict(lr=float("nan"))), EINVAL),
])
def test_adamw_list(kw, rc):
    assert _adamw(**kw) == rc
    assert "bfz_adamw_list" in bfz.lib().bfz_last_error().decode()


def test_adamw_list_null():
    f = bfz.lib().bfz_adamw_list
    assert f(None, 1, None, None, None) == EINVAL
    h = bfz.AdamW(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    assert f(None, 1, C.byref(h), None, None) == EINVAL and f(None, 0, C.byref(h), None, None) == bfz.BFZ_OK


class _Here(torch.Tensor):
    """Stands for a tensor of cuda:0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class _Elsewhere(_Here):
    def get_device(self):
        return 1


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Here)


def _forms():
    u8 = torch.uint8
    work = dict(work=_z(1 << 27, dtype=u8))
    weight = dict(weight=_z(40, 32, dtype=u8), grid=_z(1, 1))
    codes = dict(x=_z(6, 32, dtype=u8), scales=_z(1, 6))
    return [
        (bfz.quantize, dict(x=_z(6, 32), codes=_z(6, 32, dtype=u8), scales=_z(1, 6))),
        (bfz.linear, dict(out=_z(6, 40), **codes, **weight, **work)),
        (bfz.linear, dict(x=_z(6, 32), out=_z(6, 40), **weight, **work)),
        (bfz.linear_grad_input, dict(dout=_z(6, 48, dtype=u8)[:, :40], scales=_z(1, 6), dx=_z(6, 32), **weight, **work)),
        (bfz.linear_grad_weight, dict(dout=_z(6, 48, dtype=u8)[:, :40], dout_grid=_z(1, 1), x=_z(6, 32, dtype=u8), x_grid=_z(1, 1), dweight=_z(40, 32), **work)),
        (bfz.layer_norm, dict(x=_z(6, 32), weight=_z(32), bias=_z(32), out=_z(6, 32), mean=_z(6), rstd=_z(6))),
        (bfz.layer_norm_grad, dict(dout=_z(6, 32), x=_z(6, 32), weight=_z(32), mean=_z(6), rstd=_z(6), dx=_z(6, 32), dweight=_z(32), dbias=_z(32), **work)),
    ]


@pytest.fixture
def at_home(monkeypatch):
    """Device 0 is current; a call that would launch fails."""
    import sys

    from blockwise_fp8_zero_amd import _tensors
    _tensors._load()
    monkeypatch.setattr(_tensors, "_current", lambda: 0)

    def refuse(stream, home=None):
        pytest.fail("nothing may be launched")

    for name in ("linear", "layer_norm", "adamw_list"):
        monkeypatch.setattr(sys.modules[f"blockwise_fp8_zero_amd.{name}"], "raw_stream", refuse)


def test_tensors_of_another_device(at_home):
    count = 0
    for f, kw in _forms():
        for name, t in kw.items():
            with pytest.raises(ValueError, match="current device is cuda:0"):
                f(**{**kw, name: t.as_subclass(_Elsewhere)})
            count += 1
    assert count == 41


def test_shapes_and_types(at_home):
    u8 = torch.uint8
    for f, kw in _forms():
        for name, t in kw.items():
            if name in ("work", "grid"):
                bad = _z(1, dtype=u8)
            elif t.dim() == 2:
                bad = _z(t.shape[0], t.shape[1] + 16, dtype=t.dtype)
            else:
                bad = _z(t.shape[0] - 1, dtype=t.dtype)
            with pytest.raises((ValueError, TypeError)):
                f(**{**kw, name: bad})
            with pytest.raises((ValueError, TypeError)):
                f(**{**kw, name: torch.zeros(t.shape, dtype=torch.int16).as_subclass(_Here) if name != "work" else None})
    with pytest.raises(TypeError, match="scales"):
        bfz.linear(_z(6, 32, dtype=u8), _z(40, 32, dtype=u8), _z(1, 1), _z(6, 40), _z(1 << 27, dtype=u8))
    with pytest.raises(ValueError, match="16 columns"):
        bfz.quantize(_z(1, 33), _z(1, 33, dtype=u8), _z(1, 1))


def test_adamw_list_class(at_home):
    p, g = [_z(300), _z(5, 6)], [_z(300), _z(5, 6)]
    m, v, ms, vs = (list(x) for x in bfz.adamw_states([torch.zeros(300), torch.zeros(5, 6)], bits=8))
    m, v, ms, vs = ([t.as_subclass(_Here) for t in x] for x in (m, v, ms, vs))
    assert [t.numel() for t in ms] == [2, 1] and m[1].shape == (5, 6) and m[0].dtype == torch.uint8
    opt = bfz.AdamWList(p, m, v, ms, vs)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    with pytest.raises(ValueError, match="none of its own"):
        opt.step(hp)
    for bad in ([g[0]], [g[0], _z(31)], [g[0], _z(5, 12)[:, ::2]], [g[0], g[1].as_subclass(_Elsewhere)], [g[0], _z(5, 6, dtype=torch.uint8)]):
        with pytest.raises((ValueError, TypeError)):
            opt.step(hp, grads=bad)
    for args in ((p, m, v), (p, m, v, ms, vs[:1]), (p, m, [v[0], _z(30)], ms, vs), (p, m, v, [_z(3), ms[1]], vs), (p, [_z(300), m[1]], v, ms, vs),
                 (p, [_z(300), _z(30)], [_z(300), _z(30)], ms, vs)):
        with pytest.raises((ValueError, TypeError)):
            bfz.AdamWList(*args)
    with pytest.raises(ValueError):
        bfz.adamw_states(p, bits=16)


def test_refused_gradients_leave_the_list_as_it_was(at_home):
    p, g = [_z(300), _z(30)], [_z(300), _z(30)]
    opt = bfz.AdamWList(p, [_z(300), _z(30)], [_z(300), _z(30)], grads=g)
    before = list(opt._words)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    with pytest.raises(ValueError):
        opt.step(hp, grads=[_z(300, dtype=torch.bfloat16), _z(31)])
    assert list(opt._words) == before
