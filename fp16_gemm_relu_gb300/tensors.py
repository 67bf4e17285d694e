"""What the operators' torch entry points share: argument checks, streams, and the C call."""

from __future__ import annotations

import contextlib

import torch

from . import binding


def rows(t: torch.Tensor, name: str) -> int:
    """The leading dimension of a 2-D CUDA fp16 tensor of rows with unit column stride."""
    if t.dtype != torch.float16:
        raise TypeError(f"{name} must be torch.float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    n = t.shape[1]
    if n > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (unit stride along columns)")
    if t.shape[0] <= 1:
        return max(n, 1)
    ld = t.stride(0)
    if ld < max(n, 1):
        raise ValueError(f"{name}'s rows overlap")
    return ld


def param_type(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float16:
        return binding.TG_TYPE_F16
    if t.dtype == torch.float32:
        return binding.TG_TYPE_F32
    raise TypeError(f"{name} must be torch.float16 or torch.float32")


@contextlib.contextmanager
def _other_stream(device, stream, tensors):
    with torch.cuda.device(device):
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            yield stream.cuda_stream


class _Here:
    """The current stream of the current device: nothing to enter."""

    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def stream_of(device: torch.device, stream, *tensors):
    """Context that gives the handle of ``stream`` (None: torch's current one on ``device``), with
    ``device`` current.  On a stream of the caller's, outputs are allocated there and the inputs are
    kept until its work is done."""
    if stream is None and device.index == torch.cuda.current_device():
        return _Here(torch.cuda.current_stream(device).cuda_stream)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return _other_stream(device, stream, tensors)


def call(name: str, *args) -> None:
    """The C function ``name``: tensors go as pointers, None as NULL, a zero stream as NULL."""
    lib = binding._lib or binding.load_library()
    st = getattr(lib, name)(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args])
    if st != binding.TG_OK:
        raise binding.TgError(st, name)
