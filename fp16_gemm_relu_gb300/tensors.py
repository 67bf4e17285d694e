"""What the operators' torch entry points share: argument checks, streams, and the C call.

The smallest calls take a few microseconds on the GPU, so the common case (tensors of the current
device, torch's current stream) goes without context managers and temporary objects.
"""

from __future__ import annotations

import contextlib

import torch

from . import binding

_F16, _F32 = torch.float16, torch.float32


def rows(t: torch.Tensor, name: str) -> int:
    """The leading dimension of a 2-D CUDA fp16 tensor of rows with unit column stride."""
    if t.dtype is not _F16:
        raise TypeError(f"{name} must be torch.float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    m, n = t.shape
    ld, unit = t.stride()
    if unit != 1 and n > 1:
        raise ValueError(f"{name} must be row-major (unit stride along columns)")
    if m <= 1:
        return n or 1
    if ld < n or ld < 1:
        raise ValueError(f"{name}'s rows overlap")
    return ld


def param_type(t: torch.Tensor, name: str) -> int:
    if t.dtype is _F16:
        return binding.TG_TYPE_F16
    if t.dtype is _F32:
        return binding.TG_TYPE_F32
    raise TypeError(f"{name} must be torch.float16 or torch.float32")


def vector(t: torch.Tensor, n: int, index: int, name: str) -> None:
    """A dense vector of n values on the CUDA device `index`."""
    if t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous ({n},) tensor on x's device")


def written(t: torch.Tensor) -> None:
    """Tells autograd that a kernel writes to ``t``, as an in-place torch operation would.  A leaf that
    wants its gradient is refused, as there."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("out must not require a gradient: this call is not differentiable")
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def here(index: int, stream) -> bool:
    """Whether a call goes to torch's current stream of the current device."""
    return stream is None and index == _current_device()


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


@contextlib.contextmanager
def on(device: torch.device, stream, *tensors):
    """Makes ``device`` and ``stream`` (a torch stream or a handle; None: torch's current one on that
    device) current.  On a stream of the caller's, outputs are allocated there, and the inputs are
    kept until its work is done."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            yield


def _torch_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


#: Handle of torch's current stream on a device: without the Stream object where torch offers that.
stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", _torch_stream)


def ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def library():
    return binding._lib or binding.load_library()


def check(status: int, name: str) -> None:
    if status != binding.TG_OK:
        raise binding.TgError(status, name)
