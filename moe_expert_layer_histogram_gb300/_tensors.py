"""Argument checks shared by the torch wrappers, kept short: a small call's
time is mostly spent on the host."""
import torch

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_LARGEST = 2 ** 31 - 1


def fits(n, name):
    """The library takes sizes as 32-bit integers (and ctypes would cut them)."""
    if not -_LARGEST <= n <= _LARGEST:
        raise ValueError("%s: %d is beyond 2^31 - 1" % (name, n))


def stream_on(device):
    """Torch's current stream on `device`, which has to be the current one
    (the library launches on the current CUDA device)."""
    index = device.index
    if index != _current_device():
        raise ValueError("tensors on %s, current device cuda:%d" % (device, _current_device()))
    return _raw_stream(index)


def row_stride(t, dtype, name):
    """Row stride of a CUDA matrix with contiguous rows.  (Rows that overlap
    are left to the library's own check.)"""
    if t.dtype is not dtype or not t.is_cuda or t.dim() != 2:
        raise ValueError("%s: a CUDA %s matrix" % (name, dtype))
    (rows, cols), (ld, one) = t.shape, t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s: a matrix with contiguous rows" % name)
    if rows > _LARGEST or cols > _LARGEST:
        raise ValueError("%s: more than 2^31 - 1 rows or columns" % name)
    return ld if rows > 1 or ld > cols else cols


def check(t, dtype, shape, device, name):
    """A contiguous tensor of this type, shape and device, at most 2^31 - 1 in
    its first dimension."""
    if (t.dtype is not dtype or t.shape != shape or t.device != device
            or not t.is_contiguous()):
        raise ValueError("%s: contiguous %s %s on %s" % (name, dtype, tuple(shape), device))
    fits(shape[0], name)
