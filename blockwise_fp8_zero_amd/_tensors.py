"""Argument marshalling shared by the operators around the step.  Pointers are
plain integers here: at the smallest sizes a call costs what its arguments do.

Each tensor's device is compared with `home`, the device that is current at the
call's start: a kernel launched there could not follow another one's pointers.
"""
F32, BF16, F16, E4M3, F32_ROUNDED = 0, 1, 2, 3, 4

_torch = _floats = _codes = _raw = None
_ready = False
_current = None


def _load():
    """torch, on first use, and the dtype codes."""
    global _torch, _floats, _codes, _raw, _current
    if _torch is None:
        import torch
        # the handle of the current stream without a Stream object around it
        # (0.1 us instead of 2.8 of a call's 7 to 10), where torch has them
        _raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # (-2 where there is no device: a host tensor is of -1)
        _current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device) if torch.cuda.device_count() else lambda: -2
        _floats = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        _codes = {**_floats, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}
        _torch = torch
    return _torch


def home_device():
    """Index of the device that a call launches on."""
    if _current is None:
        _load()
    return _current()


def elsewhere(t, name, home):
    """Refuses what is not of the device `home`."""
    index = t.get_device() if isinstance(t, _torch.Tensor) else t.device_index
    if index < 0:
        raise TypeError(f"{name}: need a CUDA tensor")
    raise ValueError(f"{name}: is of cuda:{index}, the current device is cuda:{home}")


def raw_stream(stream, home=None):
    """hipStream_t of a torch stream of the current device, of the current one by
    default."""
    global _ready
    if home is None:
        home = home_device()
    if stream is None and _ready:
        return _raw(home)
    torch = _load()
    if stream is not None:
        if stream.device_index != home:
            elsewhere(stream, "stream", home)
        return stream.cuda_stream
    _ready = _raw is not None and torch.cuda.is_initialized()
    return torch.cuda.current_stream().cuda_stream


def dtype_code(t, name, home, codes=False):
    """BFZ_* code of a device tensor's dtype (uint8: E4M3 codes, if allowed)."""
    known = _codes if codes else _floats
    code = known.get(t.dtype) if isinstance(t, _torch.Tensor) else None
    if code is None:
        raise TypeError(f"{name}: need a CUDA tensor of {', '.join(str(x) for x in known)}")
    if t.get_device() != home:
        elsewhere(t, name, home)
    return code


def matrix(t, name, home, codes=False):
    """(pointer, dtype code, rows, columns, row stride) of a 2-D device tensor
    of unit inner stride whose rows do not overlap."""
    code = dtype_code(t, name, home, codes)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise TypeError(f"{name}: need a 2-D tensor of unit inner stride")
    rows, cols = shape
    ld = stride[0] if rows > 1 else cols
    if ld < cols:
        raise TypeError(f"{name}: rows overlap")
    return t.data_ptr(), code, rows, cols, ld


def id_vector(t, name, home):
    """(pointer, 1 for int64 or 0 for int32, count) of a contiguous id tensor."""
    torch = _torch
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.int64, torch.int32) or not t.is_contiguous():
        raise TypeError(f"{name}: need a contiguous int64 or int32 CUDA tensor")
    if t.get_device() != home:
        elsewhere(t, name, home)
    return t.data_ptr(), int(t.dtype == torch.int64), t.numel()


def vector(t, name, home, n, dtype=None):
    """Pointer of a contiguous device tensor of at least n elements (float32
    unless dtype says)."""
    torch = _torch
    want = dtype or torch.float32
    if not isinstance(t, torch.Tensor) or t.dtype != want or not t.is_contiguous():
        raise TypeError(f"{name}: need a contiguous {want} CUDA tensor")
    if t.get_device() != home:
        elsewhere(t, name, home)
    if t.numel() < n:
        raise ValueError(f"{name}: needs at least {n} elements, has {t.numel()}")
    return t.data_ptr()


def scalar(t, name, home, dtype=None):
    """Pointer of a one-element device tensor, None for None."""
    if t is None:
        return None
    p = vector(t, name, home, 1, dtype)
    if t.numel() != 1:
        raise ValueError(f"{name}: needs one element, has {t.numel()}")
    return p


def tile_grid(grid, home, code, rows, cols):
    """Pointer of an E4M3 matrix's scale grid, None for other types."""
    if code != E4M3:
        if grid is not None:
            raise ValueError("grid: only E4M3 codes have one")
        return None
    if grid is None:
        raise TypeError("grid: E4M3 codes need a contiguous float32 CUDA tensor of tile scales")
    return vector(grid, "grid", home, -(-rows // 128) * -(-cols // 128))


def work_pointer(work, home, need):
    if not isinstance(work, _torch.Tensor) or not work.is_contiguous():
        raise TypeError("work: need a contiguous CUDA tensor")
    if work.get_device() != home:
        elsewhere(work, "work", home)
    if work.numel() * work.element_size() < need:
        raise ValueError(f"work: needs at least {need} bytes, has {work.numel() * work.element_size()}")
    return work.data_ptr()
