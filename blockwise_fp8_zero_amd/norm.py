"""Global gradient norm over many tensors, and clipping (include/bfz.h:
bfz_grad_norm, bfz_shard_grad_norm, bfz_clip_coef, bfz_clip_grads).

    work = bfz.norm_workspace()                                # once
    bfz.shard_grad_norm(plan, grads, norm, work, max_norm=1.0, coef=coef)
    bfz.fold_adamw_fp8_step_unpack(plan, grads, ..., hp, grad_scale=coef)

Over several ranks: shard_grad_norm(..., sumsq=s), all_reduce(s), clip_coef(s,
1.0, norm, coef), then the step.
"""
import ctypes as C

from . import _check, _ptr_array, _weight_sizes, lib
from ._tensors import _load, dtype_code, elsewhere, home_device, raw_stream, scalar, work_pointer


def _work_bytes(_known=[]):
    if not _known:
        _known.append(int(lib().bfz_norm_work_bytes()))
    return _known[0]


def norm_workspace(device="cuda"):
    """Workspace of the norm calls: zeroed here once, then kept as they leave
    it.  Calls that may run at the same time (two streams) need one each."""
    import torch
    return torch.zeros(_work_bytes(), dtype=torch.uint8, device=device)


def _list(tensors, name, home):
    """bfz_tensor[]: three 64-bit words each (the type and a zero share one)."""
    words = []
    for t in tensors:
        code = dtype_code(t, name, home)
        if not t.is_contiguous():
            raise TypeError(f"{name}: need contiguous tensors")
        words += (t.data_ptr(), t.numel(), code)
    return (C.c_int64 * max(1, len(words)))(*words)


def _results(norm, coef, sumsq, home):
    return ((None if sumsq is None else scalar(sumsq, "sumsq", home, _load().float64)), scalar(norm, "norm", home),
            scalar(coef, "coef", home))


def _limit(max_norm):
    return float("inf") if max_norm is None else float(max_norm)


def grad_norm(grads, norm, work, max_norm=None, coef=None, sumsq=None, stream=None):
    """norm = sqrt(sum of g^2 over all of grads) and coef = min(1, max_norm /
    (norm + 1e-6)), float32 device scalars; sumsq: float64.  Each of the three
    may be None; max_norm None never clips.  grads: float32, bfloat16 or
    float16 device tensors of any shapes, mixed as they come."""
    home = home_device()
    arr = _list(grads, "grads", home)
    s, n, c = _results(norm, coef, sumsq, home)
    rc = lib().bfz_grad_norm(arr, len(grads), _limit(max_norm), s, n, c, work_pointer(work, home, _work_bytes()), raw_stream(stream, home))
    if rc:
        _check(rc)


def shard_grad_norm(plan, grads, norm, work, max_norm=None, coef=None, sumsq=None, stream=None):
    """grad_norm over the tiles the plan's rank owns, read from the row-major
    float32 gradients grads[p] (None for weights the rank does not touch)."""
    import torch
    arr = _ptr_array(grads, torch.float32, "grads", _weight_sizes(plan))
    home = home_device()
    for k, g in enumerate(grads):
        if g is not None and g.get_device() != home:
            elsewhere(g, f"grads[{k}]", home)
    s, n, c = _results(norm, coef, sumsq, home)
    _check(lib().bfz_shard_grad_norm(plan.handle, arr, _limit(max_norm), s, n, c, work_pointer(work, home, _work_bytes()),
                                     raw_stream(stream, home)))


def clip_coef(sumsq, max_norm, norm, coef, stream=None):
    """norm and coef from a device sumsq (float64), e.g. after an all-reduce."""
    home = home_device()
    s, n, c = _results(norm, coef, sumsq, home)
    _check(lib().bfz_clip_coef(s, _limit(max_norm), n, c, raw_stream(stream, home)))


def clip_grads(grads, coef, outs=None, stream=None):
    """outs[k] = grads[k] * coef, rounded once to outs[k]'s type; outs None
    clips in place."""
    outs = grads if outs is None else outs
    if len(outs) != len(grads):
        raise ValueError(f"outs: {len(outs)} tensors for {len(grads)} gradients")
    home = home_device()
    a = _list(grads, "grads", home)
    b = a if outs is grads else _list(outs, "outs", home)
    _check(lib().bfz_clip_grads(a, b, len(grads), scalar(coef, "coef", home), raw_stream(stream, home)))
