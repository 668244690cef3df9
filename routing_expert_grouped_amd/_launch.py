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
    stream and the current device is the tensors' device."""

    __slots__ = ("device", "handle", "_guards")

    def __init__(self, device: torch.device, stream=None):
        if device.type != "cuda":
            raise ValueError(f"need CUDA tensors, got {device}")
        self.device = device
        self._guards = ()
        if device.index != torch.cuda.current_device():
            self._guards = (torch.cuda.device(device),)
        if stream is None:
            self.handle = torch.cuda.current_stream(device).cuda_stream
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
        self._check(t, name, dtype)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous tensor")
        return t.data_ptr()

    def rows(self, t, name, dtype, cols, nrows=None):
        """(pointer, row pitch, rows) of a 2-D tensor whose rows are contiguous; the rows may be
        further apart than they are long (a column slice of a wider tensor)."""
        self._check(t, name, dtype)
        if t.dim() != 2 or t.shape[1] != cols or (nrows is not None and t.shape[0] != nrows):
            want = ("rows" if nrows is None else nrows, cols)
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {want}")
        n, ld = t.shape[0], t.stride(0)
        if n <= 1:
            ld = max(ld, cols)
        if (cols > 1 and t.stride(1) != 1) or ld < cols:
            raise ValueError(f"{name}: strides {t.stride()}: need contiguous rows that do not "
                             "overlap")
        return t.data_ptr(), ld, n

    def buffer(self, t, name, nbytes):
        """Pointer of a contiguous buffer of at least nbytes bytes."""
        self._check(t, name, t.dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name}: need a contiguous tensor")
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"{name}: {have} bytes, the shape needs {nbytes}")
        return t.data_ptr()

    def _check(self, t, name, dtype):
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, expected {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def elt16(t, name):
    """The 16-bit element type of a tensor, as the C enum."""
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16 or float16")
    return ELT[t.dtype]
