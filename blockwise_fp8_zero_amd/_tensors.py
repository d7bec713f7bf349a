"""Argument marshalling shared by the operators around the step."""
import ctypes as C

F32, BF16, F16, E4M3 = 0, 1, 2, 3


def dtype_code(t, name, codes=False):
    """BFZ_* code of a device tensor's dtype (uint8: E4M3 codes, if allowed)."""
    import torch
    types = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    if codes:
        types.update({torch.uint8: E4M3, torch.float8_e4m3fn: E4M3})
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in types:
        raise TypeError(f"{name}: need a CUDA tensor of {', '.join(str(x) for x in types)}")
    return types[t.dtype]


def matrix(t, name, codes=False):
    """(pointer, dtype code, rows, columns, row stride) of a 2-D device tensor
    of unit inner stride whose rows do not overlap."""
    code = dtype_code(t, name, codes)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise TypeError(f"{name}: need a 2-D tensor of unit inner stride")
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise TypeError(f"{name}: rows overlap")
    return C.c_void_p(t.data_ptr()), code, rows, cols, ld


def id_vector(t, name):
    """(pointer, 1 for int64 or 0 for int32, count) of a contiguous id tensor."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in (torch.int64, torch.int32) or not t.is_contiguous():
        raise TypeError(f"{name}: need a contiguous int64 or int32 CUDA tensor")
    return C.c_void_p(t.data_ptr()), int(t.dtype == torch.int64), t.numel()


def tile_grid(grid, code, rows, cols):
    """Pointer of an E4M3 matrix's scale grid, None for other types."""
    import torch
    if code != E4M3:
        if grid is not None:
            raise ValueError("grid: only E4M3 codes have one")
        return None
    need = -(-rows // 128) * -(-cols // 128)
    if (not isinstance(grid, torch.Tensor) or not grid.is_cuda or grid.dtype != torch.float32
            or not grid.is_contiguous()):
        raise TypeError("grid: E4M3 codes need a contiguous float32 CUDA tensor of tile scales")
    if grid.numel() < need:
        raise ValueError(f"grid: needs at least {need} elements, has {grid.numel()}")
    return C.c_void_p(grid.data_ptr())


def work_pointer(work, need):
    import torch
    if not isinstance(work, torch.Tensor) or not work.is_cuda or not work.is_contiguous():
        raise TypeError("work: need a contiguous CUDA tensor")
    if work.numel() * work.element_size() < need:
        raise ValueError(f"work: needs at least {need} bytes, has {work.numel() * work.element_size()}")
    return C.c_void_p(work.data_ptr())
