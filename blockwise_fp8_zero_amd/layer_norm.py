"""Layer norm and its gradient (include/bfz.h: bfz_layer_norm,
bfz_layer_norm_grad)."""
from . import _check, lib
from ._tensors import dtype_code, home_device, matrix, raw_stream, vector, work_pointer


def _params(home, dim, **tensors):
    """Pointers of vectors of dim elements (None for None) and their common
    dtype code, float32's where there is none."""
    code, out = None, []
    for name, t in tensors.items():
        if t is None:
            out.append(None)
            continue
        c = dtype_code(t, name, home)
        if code is not None and c != code:
            raise TypeError(f"{', '.join(tensors)}: need one dtype")
        code = c
        if not t.is_contiguous() or t.numel() != dim:
            raise ValueError(f"{name}: need {dim} contiguous elements")
        out.append(t.data_ptr())
    return out, code or 0


def _same(t, name, home, shape):
    p, code, rows, cols, ld = matrix(t, name, home)
    if (rows, cols) != shape:
        raise ValueError(f"{name}: is {(rows, cols)}, need {shape}")
    return p, code, ld


def layer_norm(x, weight, bias, out, eps=1e-5, mean=None, rstd=None, stream=None):
    """out = (x - mean) rstd weight + bias over the rows of x (n, dim); weight,
    bias: dim elements of one dtype, each may be None; mean, rstd: float32 (n),
    for layer_norm_grad, each may be None.  x, out: float32, bfloat16 or float16."""
    home = home_device()
    p, code, n, dim, ld = matrix(x, "x", home)
    (w, b), pcode = _params(home, dim, weight=weight, bias=bias)
    o, ocode, old = _same(out, "out", home, (n, dim))
    rc = lib().bfz_layer_norm(p, code, ld, n, dim, w, b, pcode, eps, o, ocode, old, None if mean is None else vector(mean, "mean", home, n),
                              None if rstd is None else vector(rstd, "rstd", home, n), raw_stream(stream, home))
    if rc:
        _check(rc)


def layer_norm_workspace(n, dim, device="cuda"):
    """Workspace of layer_norm_grad for up to n rows."""
    import torch
    return torch.empty(max(256, int(lib().bfz_layer_norm_work_bytes(int(n), int(dim)))), dtype=torch.uint8, device=device)


def layer_norm_grad(dout, x, weight, mean, rstd, dx, dweight, dbias, work, accumulate=False, stream=None):
    """dx (n, dim), dweight and dbias (dim elements of one dtype) from dout (n,
    dim); each of the three may be None, and so may work where dweight and dbias
    are.  mean, rstd: as layer_norm wrote them.  accumulate adds to dweight and
    dbias."""
    home = home_device()
    p, code, n, dim, ld = matrix(x, "x", home)
    d, dcode, dld = _same(dout, "dout", home, (n, dim))
    (w,), pcode = _params(home, dim, weight=weight)
    (dw, db), gcode = _params(home, dim, dweight=dweight, dbias=dbias)
    o, ocode, old = (None, 0, dim) if dx is None else _same(dx, "dx", home, (n, dim))
    wp = None
    if work is not None or dw is not None or db is not None:
        wp = work_pointer(work, home, lib().bfz_layer_norm_work_bytes(n, dim))
    rc = lib().bfz_layer_norm_grad(d, dcode, dld, p, code, ld, n, dim, w, pcode, vector(mean, "mean", home, n),
                                   vector(rstd, "rstd", home, n), o, ocode, old, dw, db, gcode, int(bool(accumulate)), wp,
                                   raw_stream(stream, home))
    if rc:
        _check(rc)
