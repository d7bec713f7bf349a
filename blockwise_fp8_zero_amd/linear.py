"""The linear layer in E4M3 on the row-major FP8 weights and scale grids that the
step writes, its gradients, and the quantizer of its activations (include/bfz.h:
bfz_quantize, bfz_linear, bfz_linear_grad_input, bfz_linear_grad_weight).

    codes, grid = bfz.quantize_buffers(n, cols, tiles=True)        # once
    work = bfz.linear_workspace(n, weight)
    bfz.quantize(x, codes, grid, tiles=True)
    bfz.linear(codes, weight, w_grid, y, work, scales=grid, tiles=True)
    ...                                                            # dy likewise: dcodes, dgrid
    bfz.linear_grad_input(dcodes, weight, w_grid, dx, work, scales=dgrid, tiles=True)
    bfz.linear_grad_weight(dcodes, dgrid, codes, grid, dweight, work)

Without gradients, bfz.linear(x, weight, w_grid, y, work) quantizes x itself.
"""
from . import _check, lib
from . import _tensors
from ._tensors import BF16, BF16_EXACT, E4M3, home_device, matrix, raw_stream, tile_grid, work_pointer


def quantize_buffers(n, dim, tiles=False, device="cuda"):
    """Codes (n, dim) and scales for quantize: the codes' rows start on 16-byte
    boundaries; scales (ceil(dim/128), n) of row groups or the grid
    (ceil(n/128), ceil(dim/128)) of tiles."""
    import torch
    codes = torch.zeros((max(1, n), -(-dim // 16) * 16), dtype=torch.uint8, device=device)[:n, :dim]
    shape = (-(-n // 128), -(-dim // 128)) if tiles else (-(-dim // 128), n)
    return codes, torch.empty(shape, dtype=torch.float32, device=device)


def _rows(t, name, home):
    """(pointer, rows, columns, row stride) of codes whose rows are read and
    written up to the next multiple of 16 columns."""
    p, code, rows, cols, ld = matrix(t, name, home, codes=True)
    if code != E4M3:
        raise TypeError(f"{name}: need E4M3 codes (uint8)")
    if cols & 15 and rows:
        wide = -(-cols // 16) * 16
        if rows == 1:
            ld = wide  # a single row's stride says nothing
        if t.storage_offset() + (rows - 1) * ld + wide > t.untyped_storage().nbytes():
            raise ValueError(f"{name}: rows have to reach to the next multiple of 16 columns (see quantize_buffers)")
    return p, rows, cols, ld


def _scales(t, name, home, n, dim, tiles):
    """(pointer, row stride) of the scales of (n, dim) codes."""
    p, code, rows, cols, ld = matrix(t, name, home)
    if code or (rows, cols) != ((-(-n // 128), -(-dim // 128)) if tiles else (-(-dim // 128), n)):
        raise ValueError(f"{name}: need float32 {(-(-n // 128), -(-dim // 128)) if tiles else (-(-dim // 128), n)}")
    return p, ld


def quantize(x, codes, scales, tiles=False, pow2=False, stream=None):
    """codes, scales = E4M3 form of x, one scale for each 128 columns of a row
    (scales: (ceil(dim/128), n)) or for each 128x128 tile (tiles=True; scales:
    (ceil(n/128), ceil(dim/128))); pow2: scales are powers of two.  x: (n, dim)
    float32, bfloat16 or float16; codes: uint8 (n, dim), rows on 16-byte
    boundaries (quantize_buffers)."""
    home = home_device()
    p, code, n, dim, ld = matrix(x, "x", home)
    c, rows, cols, cld = _rows(codes, "codes", home)
    if (rows, cols) != (n, dim):
        raise ValueError(f"codes: is {(rows, cols)}, need {(n, dim)}")
    s, sld = _scales(scales, "scales", home, n, dim, tiles)
    rc = lib().bfz_quantize(p, code, ld, n, dim, int(bool(tiles)), int(bool(pow2)), c, cld, s, sld, raw_stream(stream, home))
    if rc:
        _check(rc)


_bytes = {}  # of workspaces, by sizes


def _work_bytes(*sizes):
    need = _bytes.get(sizes)
    if need is None:
        if len(_bytes) > 4096:
            _bytes.clear()
        need = _bytes[sizes] = int(lib().bfz_linear_work_bytes(*sizes))
    return need


def linear_workspace(n, weight, x_dtype=None, device=None):
    """Workspace of linear and its gradients for up to n tokens and this weight;
    x_dtype: of inputs that linear quantizes itself (None: codes)."""
    import torch
    _tensors._load()
    rows, cols = weight.shape
    code = E4M3 if x_dtype is None else _tensors._codes.get(x_dtype)
    if code is None:
        raise TypeError(f"x_dtype: {x_dtype} is none of {', '.join(str(x) for x in _tensors._codes)}")
    copy = (weight.data_ptr() | (weight.stride(0) if rows > 1 else 0)) & 15
    need = _work_bytes(int(n), rows, cols, code, int(copy != 0))
    return torch.empty(max(256, need), dtype=torch.uint8, device=weight.device if device is None else device)


def _weight(weight, grid, home):
    """(pointer, row stride, pointer of the grid, rows, columns, whether the rows
    are copied)"""
    w, code, rows, cols, ld = matrix(weight, "weight", home, codes=True)
    if code != E4M3:
        raise TypeError("weight: need E4M3 codes (uint8)")
    return w, ld, tile_grid(grid, home, code, rows, cols), rows, cols, int(((w | ld) & 15) != 0)


def _result(t, name, home, shape, exact):
    p, code, rows, cols, ld = matrix(t, name, home)
    if (rows, cols) != shape:
        raise ValueError(f"{name}: is {(rows, cols)}, need {shape}")
    return p, BF16_EXACT if exact and code == BF16 else code, ld


def linear(x, weight, grid, out, work, scales=None, tiles=False, stream=None, exact=False):
    """out = X W^T.  x: (n, cols) E4M3 codes with the scales that quantize gave
    them (tiles: as there), or float32, bfloat16 or float16 values, which are
    quantized by rows; weight: (rows, cols) E4M3 codes with their tile scales
    `grid`; out: (n, rows) float32, bfloat16 or float16.  exact: a bfloat16 result
    of more than 16 tokens of exact products too, at half the rate (others are)."""
    home = home_device()
    p, code, n, dim, ld = matrix(x, "x", home, codes=True)
    w, wld, g, rows, cols, copy = _weight(weight, grid, home)
    if code == E4M3:
        if dim & 15 or n == 1:
            p, n, dim, ld = _rows(x, "x", home)
        if scales is None:
            raise TypeError("scales: E4M3 codes need theirs")
        s, sld = _scales(scales, "scales", home, n, dim, tiles)
    else:
        if scales is not None or tiles:
            raise ValueError("scales, tiles: only E4M3 codes have them")
        s, sld = None, 0
    if dim != cols:
        raise ValueError(f"x is {(n, dim)}, weight {(rows, cols)}")
    o, ocode, old = _result(out, "out", home, (n, rows), exact)
    rc = lib().bfz_linear(p, code, ld, s, sld, int(bool(tiles)), n, w, wld, g, rows, cols, o, ocode, old,
                          work_pointer(work, home, _work_bytes(n, rows, cols, code, copy)), raw_stream(stream, home))
    if rc:
        _check(rc)


def linear_grad_input(dout, weight, grid, dx, work, scales, tiles=False, accumulate=False, stream=None, exact=False):
    """dx = dOut W, or with accumulate added to dx.  dout: (n, rows) E4M3 codes
    with the scales that quantize gave them; dx: (n, cols) float32, bfloat16 or
    float16; exact: as for linear, whatever n is."""
    home = home_device()
    w, wld, g, rows, cols, copy = _weight(weight, grid, home)
    p, n, dim, ld = _rows(dout, "dout", home)
    if dim != rows:
        raise ValueError(f"dout is {(n, dim)}, weight {(rows, cols)}")
    s, sld = _scales(scales, "scales", home, n, dim, tiles)
    o, ocode, old = _result(dx, "dx", home, (n, cols), exact)
    rc = lib().bfz_linear_grad_input(p, ld, s, sld, int(bool(tiles)), n, w, wld, g, rows, cols, o, ocode, old, int(bool(accumulate)),
                                     work_pointer(work, home, _work_bytes(n, rows, cols, E4M3, copy)), raw_stream(stream, home))
    if rc:
        _check(rc)


def linear_grad_weight(dout, dout_grid, x, x_grid, dweight, work, accumulate=False, stream=None, exact=False):
    """dweight = dOut^T X, or with accumulate added to dweight.  dout: (n, rows)
    and x: (n, cols), E4M3 codes with their tile scales (quantize, tiles=True);
    dweight: (rows, cols) float32, bfloat16 or float16; exact: as for linear,
    whatever n is."""
    home = home_device()
    p, n, rows, ld = _rows(dout, "dout", home)
    q, count, cols, qld = _rows(x, "x", home)
    if count != n:
        raise ValueError(f"dout is {(n, rows)}, x {(count, cols)}")
    s, sld = _scales(dout_grid, "dout_grid", home, n, rows, True)
    t, tld = _scales(x_grid, "x_grid", home, n, cols, True)
    o, ocode, old = _result(dweight, "dweight", home, (rows, cols), exact)
    rc = lib().bfz_linear_grad_weight(p, ld, s, sld, q, qld, t, tld, n, rows, cols, o, ocode, old, int(bool(accumulate)),
                                      work_pointer(work, home, _work_bytes(n, rows, cols, E4M3, 0)), raw_stream(stream, home))
    if rc:
        _check(rc)
