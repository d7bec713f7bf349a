"""AdamW over many tensors at once, states in 32 or 8 bits (include/bfz.h:
bfz_adamw_list): for the norms, biases and other tensors that no shard of FP8
tiles holds.

    m, v, m_scale, v_scale = bfz.adamw_states(params, bits=8)     # zero states
    opt = bfz.AdamWList(params, m, v, m_scale, v_scale, grads=grads)
    opt.step(bfz.AdamW(lr=1e-4, ..., step=t), grad_scale=coef)
"""
import ctypes as C

from . import _check, _hparams, lib
from ._tensors import E4M3, F32, _load, dtype_code, elsewhere, home_device, raw_stream, scalar

BLOCK = 256  # elements that share the scales of 8-bit states
_WORDS = 9   # 64-bit words of a bfz_adamw_tensor


def adamw_states(params, bits=32):
    """Zero states for AdamWList: lists m, v, m_scale, v_scale, the scales None
    for 32 bits.  bits=8: E4M3 codes of m and of sqrt(v), one scale for each 256
    elements."""
    import torch
    if bits not in (8, 32):
        raise ValueError(f"bits: {bits} is neither 8 nor 32")
    dtype = torch.float32 if bits == 32 else torch.uint8
    m, v = ([torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params] for _ in range(2))
    if bits == 32:
        return m, v, [None] * len(m), [None] * len(m)
    ms, vs = ([torch.ones(-(-p.numel() // BLOCK), dtype=torch.float32, device=p.device) for p in params] for _ in range(2))
    return m, v, ms, vs


class AdamWList:
    """Tensors and their states, marshalled once.  params: float32, bfloat16 or
    float16; m, v: float32, or E4M3 codes (uint8) of m and of sqrt(v) with their
    block scales m_scale, v_scale; grads: gradients that every step reads, where
    they stay in place.  All contiguous and of one device.  The tensors are kept
    here; storage that a caller replaces needs a new list."""

    def __init__(self, params, m, v, m_scale=None, v_scale=None, grads=None):
        _load()
        none = [None] * len(params)
        lists = [list(x) for x in (params, m, v, m_scale or none, v_scale or none)]
        if any(len(x) != len(params) for x in lists):
            raise ValueError(f"m, v, m_scale, v_scale: need {len(params)} of each")
        self.params, self.m, self.v, self.m_scale, self.v_scale = lists
        self._home = self.params[0].get_device() if params else home_device()
        self._words = (C.c_int64 * max(1, _WORDS * len(params)))()
        for k, (p, a, b, sa, sb) in enumerate(zip(*lists)):
            n = p.numel() if hasattr(p, "numel") else 0
            code = self._array(p, "params", k, n)
            state = self._array(a, "m", k, n, codes=True)
            if state not in (F32, E4M3) or self._array(b, "v", k, n, codes=True) != state:
                raise TypeError(f"m[{k}], v[{k}]: need float32 or E4M3 codes, of one dtype")
            for s, name in ((sa, "m_scale"), (sb, "v_scale")):
                if (s is None) != (state == F32):
                    raise TypeError(f"{name}[{k}]: E4M3 states need their block scales, float32 states have none")
                if s is not None and self._array(s, name, k, -(-n // BLOCK)) != F32:
                    raise TypeError(f"{name}[{k}]: need float32")
            self._words[_WORDS * k:_WORDS * (k + 1)] = (p.data_ptr(), 0, a.data_ptr(), b.data_ptr(), 0 if sa is None else sa.data_ptr(),
                                                        0 if sb is None else sb.data_ptr(), n, code, state)
        self._codes = [self._words[_WORDS * k + 7] for k in range(len(params))]
        self.grads = None
        if grads is not None:
            self._put(grads, self._words)
            self.grads = list(grads)

    def _array(self, t, name, k, n, codes=False):
        code = dtype_code(t, f"{name}[{k}]", self._home, codes)
        if not t.is_contiguous():
            raise TypeError(f"{name}[{k}]: need a contiguous tensor")
        if t.numel() != n:
            raise ValueError(f"{name}[{k}]: has {t.numel()} elements, needs {n}")
        return code

    def _put(self, grads, words):
        """The gradients' pointers and types into a table."""
        if len(grads) != len(self.params):
            raise ValueError(f"grads: {len(grads)} tensors for {len(self.params)}")
        codes = [self._array(g, "grads", k, words[_WORDS * k + 6]) for k, g in enumerate(grads)]
        for k, (g, code) in enumerate(zip(grads, codes)):
            words[_WORDS * k + 1] = g.data_ptr()
            words[_WORDS * k + 7] = self._codes[k] | (code << 32)

    def step(self, hp, grads=None, grad_scale=None, stream=None):
        """One step: hp, an AdamW or a dict of its fields; grads: float32,
        bfloat16 or float16, those of the list by default; grad_scale: a float32
        device scalar that they are multiplied by (grad_norm's coef)."""
        home = home_device()
        if self._home != home and self.params:
            elsewhere(self.params[0], "params", home)
        words = self._words
        if grads is not None:
            # a table of this call's own: another thread may be in a step of its own
            words = type(words).from_buffer_copy(words)
            self._put(grads, words)
        elif self.grads is None:
            raise ValueError("grads: the list has none of its own")
        rc = lib().bfz_adamw_list(words, len(self.params), C.byref(_hparams(hp)), scalar(grad_scale, "grad_scale", home),
                                  raw_stream(stream, home))
        if rc:
            _check(rc)
