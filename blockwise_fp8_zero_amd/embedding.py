"""Token embedding and its gradient (include/bfz.h: bfz_embed,
bfz_embed_grad).  The table may be the row-major FP8 weight and scale grid
that the step writes; the gradient is the row-major one the step reads.
"""
from . import _check, lib
from ._tensors import home_device, id_vector, matrix, raw_stream, tile_grid, work_pointer


def _same(name, got, want):
    if tuple(got) != tuple(want):
        raise ValueError(f"{name}: is {tuple(got)}, need {tuple(want)}")


def embed(ids, table, out, scale=1.0, grid=None, stream=None):
    """out[k] = scale * table[ids[k]]; a zero row for an id outside the table.
    ids: int64 or int32, any shape; table: (vocab, dim) float32, bfloat16,
    float16, or E4M3 codes (uint8) with their tile scales `grid`; out:
    (ids.numel(), dim) float32, bfloat16 or float16.  Rows may be strided."""
    home = home_device()
    p, wide, n = id_vector(ids, "ids", home)
    t, tcode, vocab, dim, tld = matrix(table, "table", home, codes=True)
    o, ocode, rows, cols, old = matrix(out, "out", home)
    _same("out", (rows, cols), (n, dim))
    _check(lib().bfz_embed(p, wide, n, t, tcode, tile_grid(grid, home, tcode, vocab, dim), vocab, dim, tld, float(scale),
                           o, ocode, old, raw_stream(stream, home)))


def embed_grad_workspace(n, dim, device="cuda"):
    """Workspace of embed_grad for up to n tokens of width dim."""
    import torch
    return torch.empty(max(16, int(lib().bfz_embed_grad_work_bytes(int(n), int(dim)))), dtype=torch.uint8, device=device)


def embed_grad(ids, dout, dtable, work, scale=1.0, accumulate=False, stream=None):
    """dtable[v] = scale * sum of dout[k] over ids[k] = v, in ascending k; with
    accumulate the sums are added to dtable and other rows left alone.  dout:
    (ids.numel(), dim), dtable: (vocab, dim); float32, bfloat16 or float16."""
    home = home_device()
    p, wide, n = id_vector(ids, "ids", home)
    d, dcode, rows, dim, dld = matrix(dout, "dout", home)
    t, tcode, vocab, cols, tld = matrix(dtable, "dtable", home)
    _same("dout", (rows, dim), (n, cols))
    need = lib().bfz_embed_grad_work_bytes(n, dim)
    _check(lib().bfz_embed_grad(p, wide, n, d, dcode, dld, vocab, dim, float(scale), int(bool(accumulate)), t, tcode,
                                tld, work_pointer(work, home, need), raw_stream(stream, home)))
