"""What the bindings of the products and norms share: the device and stream a call runs on, and the
checks of its tensors.

A call runs on the device of its tensors, whatever the current device is, and on the current stream
of that device unless a stream is given; buffers the binding allocates are allocated on that stream.
"""
from __future__ import annotations

import torch

from ._lib import MOE_ELT_BF16, MOE_ELT_F32, MOE_ELT_FP16

ELT = {torch.bfloat16: MOE_ELT_BF16, torch.float16: MOE_ELT_FP16, torch.float32: MOE_ELT_F32}


class Launch:
    """Context of one call: `handle` is the hipStream_t; inside it, allocations belong to that
    stream and the current device is the tensors' device. (A call on the current device and stream,
    the usual one, enters nothing: the checks are a good part of a small call's time.)"""

    __slots__ = ("device", "index", "handle", "_guards")

    def __init__(self, device: torch.device, stream=None):
        if device.type != "cuda":
            raise ValueError(f"need CUDA tensors, got {device}")
        self.device = device
        self.index = device.index
        self._guards = ()
        if self.index != torch.cuda.current_device():
            self._guards = (torch.cuda.device(device),)
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            if stream.device != device:
                raise ValueError(f"stream on {stream.device}, tensors on {device}")
            self.handle = stream.cuda_stream
            self._guards += (torch.cuda.stream(stream),)

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return self

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False

    def empty(self, *shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def dense(self, t, name, dtype, *shape):
        """Pointer of a contiguous tensor of this dtype and shape on the call's device; None is
        None."""
        if t is None:
            return None
        if t.dtype is not dtype or t.get_device() != self.index:
            self._refuse(t, name, dtype)
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous tensor")
        return t.data_ptr()

    def rows(self, t, name, dtype, cols, nrows=None):
        """(pointer, row pitch, rows) of a 2-D tensor whose rows are contiguous; the rows may be
        further apart than they are long (a column slice of a wider tensor)."""
        if t.dtype is not dtype or t.get_device() != self.index:
            self._refuse(t, name, dtype)
        shape = t.shape
        if len(shape) != 2 or shape[1] != cols or (nrows is not None and shape[0] != nrows):
            want = ("rows" if nrows is None else nrows, cols)
            raise ValueError(f"{name}: shape {tuple(shape)}, expected {want}")
        n = shape[0]
        ld, step = t.stride()
        if n <= 1:
            ld = max(ld, cols)
        if (cols > 1 and step != 1) or ld < cols:
            raise ValueError(f"{name}: strides {t.stride()}: need contiguous rows that do not "
                             "overlap")
        return t.data_ptr(), ld, n

    def buffer(self, t, name, nbytes):
        """Pointer of a contiguous buffer of at least nbytes bytes."""
        if t.get_device() != self.index:
            self._refuse(t, name, t.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous tensor")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"{name}: {have} bytes, the shape needs {nbytes}")
        return t.data_ptr()

    def _refuse(self, t, name, dtype):
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, expected {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def elt16(t, name):
    """The 16-bit element type of a tensor, as the C enum."""
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16 or float16")
    return ELT[t.dtype]
