"""What the wrappers of the newer entry points share: argument checks, the
stream and device of a call, and the status word of calls that return none."""
from __future__ import annotations

import contextlib
import struct

import torch

from . import _binding as B

_status: dict[int, torch.Tensor] = {}

# The handle of a device's current stream without a torch.cuda.Stream around
# it, whose making takes 2 us: a fifth of a small call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return B.MOE_BF16
    if t == torch.float32:
        return B.MOE_F32
    raise TypeError(f"unsupported dtype {t}: bfloat16 or float32 is needed")


def record(n):
    """Packs n numbers (pointers, sizes, flags) for a moe_bind_* function."""
    return struct.Struct(f"{n}q").pack


def ptr(t):
    return None if t is None else t.data_ptr()


def need(name, t, dtype, shape, dev):
    """Raises unless t is a contiguous tensor of this type, shape and device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or not t.is_contiguous() \
            or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {dev}"
                         + ("" if shape is None else f" of shape {tuple(shape)}"))


def cuda(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the kernels run only on the GPU)")
    return t.device


@contextlib.contextmanager
def _scope(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield _raw_stream(dev.index)
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream, device=dev)
            with torch.cuda.stream(s):
                yield s.cuda_stream


class on:
    """The device and stream of a call, as its stream handle. What the call
    allocates inside belongs to that stream, so memory that it lets go is not
    handed out again before the kernels that use it. stream: None (torch's
    current one), a torch.cuda.Stream or a cudaStream_t as an integer."""

    def __init__(self, dev, stream):
        # the ordinary call (current device and stream) goes without contexts
        self._plain = stream is None and torch.cuda.current_device() == dev.index
        self._dev = dev
        self._ctx = None if self._plain else _scope(dev, stream)

    def __enter__(self):
        return _raw_stream(self._dev.index) if self._plain else self._ctx.__enter__()

    def __exit__(self, *exc):
        return None if self._plain else self._ctx.__exit__(*exc)


def device_status(dev) -> torch.Tensor:
    """The status word ([1] int32) of a device, into which ``mx_matmul`` calls
    that are given none OR their MOE_DEV_* bits, on every stream and thread: it
    says that some call since it was last cleared had a fault, not which one.
    Read it after synchronising; the caller clears it. The first use on a device
    makes it and cannot be captured into a graph."""
    if not isinstance(dev, torch.device):
        dev = torch.device(dev)
    i = torch.cuda.current_device() if dev.index is None else dev.index
    if i not in _status:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first call on a device must not be captured into a graph: its status word would "
                               "belong to the graph (call once before, or pass status)")
        with torch.cuda.device(i):
            _status[i] = torch.zeros((1,), dtype=torch.int32, device=f"cuda:{i}")
            torch.cuda.current_stream().synchronize()  # cleared before a call on any stream
    return _status[i]


def check(st, lib):
    if st != B.MOE_OK:
        raise B.MoEError(st, B.last_error_detail(lib))

