"""Softmax cross entropy over a large vocabulary, and its gradient, without
the logits in memory (include/bfz.h: bfz_vocab_loss, bfz_vocab_loss_grad).  The
head's weight may be the row-major FP8 weight and scale grid that the step
writes.
"""
from . import _check, lib
from ._tensors import BF16, E4M3, F32, F32_ROUNDED, home_device, id_vector, matrix, raw_stream, tile_grid, vector, work_pointer


def vocab_loss_workspace(n, vocab, dim, weight_dtype=None, grad=True, device="cuda"):
    """Workspace of vocab_loss and, with grad, vocab_loss_grad for up to n tokens.
    weight_dtype: torch.bfloat16, or torch.uint8 (the default) for E4M3 codes."""
    import torch
    code = BF16 if weight_dtype == torch.bfloat16 else E4M3
    need = int(lib().bfz_vocab_loss_work_bytes(int(n), int(vocab), int(dim), code, int(bool(grad))))
    return torch.empty(max(16, need), dtype=torch.uint8, device=device)


def _operands(hidden, weight, targets, grid, home):
    h, hcode, n, dim, hld = matrix(hidden, "hidden", home)
    w, wcode, vocab, cols, wld = matrix(weight, "weight", home, codes=True)
    t, wide, count = id_vector(targets, "targets", home)
    if hcode != BF16 or wcode not in (BF16, E4M3):
        raise TypeError("hidden: need bfloat16; weight: bfloat16 or E4M3 codes")
    if cols != dim or count != n:
        raise ValueError(f"hidden is {(n, dim)}, weight {(vocab, cols)}, targets {count}")
    return [h, hld, n, w, wcode, wld, tile_grid(grid, home, wcode, vocab, dim), vocab, dim, t, wide], n, vocab, dim, wcode


def _work(work, home, n, vocab, dim, wcode, grad):
    return work_pointer(work, home, lib().bfz_vocab_loss_work_bytes(n, vocab, dim, wcode, grad))


def vocab_loss(hidden, weight, targets, loss, lse, work, grid=None, stream=None):
    """loss[k] = lse[k] - z[k, targets[k]] and lse[k] = log sum exp z[k] with
    z = hidden weight^T; loss 0 for a target outside the vocabulary.  hidden:
    (n, dim) bfloat16; weight: (vocab, dim) bfloat16, or E4M3 codes (uint8) with
    their tile scales `grid`; targets: int64 or int32; loss, lse: float32 (n)."""
    home = home_device()
    args, n, vocab, dim, wcode = _operands(hidden, weight, targets, grid, home)
    _check(lib().bfz_vocab_loss(*args, vector(loss, "loss", home, n), vector(lse, "lse", home, n),
                                _work(work, home, n, vocab, dim, wcode, 0), raw_stream(stream, home)))


def vocab_loss_grad(hidden, weight, targets, lse, dloss, dhidden, dweight, work, grid=None, accumulate=False,
                    stream=None, rounded=False):
    """Gradient of sum(dloss * loss): dhidden (n, dim) bfloat16 and dweight
    (vocab, dim) bfloat16 or float32, each may be None.  lse: as vocab_loss
    wrote it; dloss: float32 (n).  accumulate adds to dweight.  A float32 dweight
    is made of the logits' gradients in two bfloat16 parts (2^-16 off at most);
    rounded=True rounds them to bfloat16 once (2^-8), in less time."""
    home = home_device()
    args, n, vocab, dim, wcode = _operands(hidden, weight, targets, grid, home)
    dh = dw = (None, 0, 0, 0, 0)
    if dhidden is not None:
        dh = matrix(dhidden, "dhidden", home)
        if dh[1] != BF16 or dh[2:4] != (n, dim):
            raise ValueError(f"dhidden: need bfloat16 {(n, dim)}")
    if dweight is not None:
        dw = matrix(dweight, "dweight", home)
        if dw[1] not in (BF16, F32) or dw[2:4] != (vocab, dim):
            raise ValueError(f"dweight: need bfloat16 or float32 {(vocab, dim)}")
    dtype = dw[1]
    if rounded:
        if dweight is None or dtype != F32:
            raise ValueError("rounded: only of a float32 dweight")
        dtype = F32_ROUNDED
    _check(lib().bfz_vocab_loss_grad(*args, vector(lse, "lse", home, n), vector(dloss, "dloss", home, n),
                                     dh[0], dh[4], dw[0], dtype, dw[4], int(bool(accumulate)),
                                     _work(work, home, n, vocab, dim, wcode, 1), raw_stream(stream, home)))
