"""Gradients unscaled and clipped by their global norm, over the C ABI (tg_clip_gradients).

Squares are summed in float32 by blocks, the blocks' sums in float64; results are the same run to run.
Calls run on ``stream`` (default: torch's current stream) and return without synchronising: the norm
stays on the device.
"""

from __future__ import annotations

import array

import torch

from .tensors import check, here, library, on, param_type, stream_handle, written


def _dense(t, name):
    """Whether t's values fill its memory without gaps, in any order of dimensions."""
    if t.is_contiguous():
        return
    n = 1
    for stride, size in sorted((s, d) for s, d in zip(t.stride(), t.shape) if d != 1):
        if stride != n:
            raise ValueError(f"{name} must fill its memory without gaps or overlaps")
        n *= size


def _clip(grads, outs, loss_scale, max_norm, stream):
    dev = grads[0].get_device()
    norm = torch.empty((), dtype=torch.float32, device=grads[0].device)
    words = []
    for i, g in enumerate(grads):
        kind = param_type(g, f"grads[{i}]")
        if g.get_device() != dev:
            raise ValueError("the gradients must be on one CUDA device")
        _dense(g, f"grads[{i}]")
        out = 0
        out_kind = 0
        if outs is not None:
            out, out_kind = outs[i].data_ptr(), param_type(outs[i], f"out[{i}]")
        words += (g.data_ptr(), out, g.numel(), kind | out_kind << 32)
    table = array.array("Q", words)
    check(library().tg_clip_gradients(table.buffer_info()[0], len(grads), loss_scale, max_norm,
                                      norm.data_ptr(), stream_handle(dev)), "tg_clip_gradients")
    return norm


def _gradients(grads):
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    if not all(g.is_cuda for g in grads):
        raise ValueError("the gradients must be CUDA tensors")
    return grads


def gradient_norm(grads, loss_scale: float = 1.0, stream=None):
    """The norm of all of ``grads`` together over ``loss_scale``, a float32 scalar on their device."""
    grads = _gradients(grads)
    if not here(grads[0].get_device(), stream):
        with on(grads[0].device, stream, *grads):
            return _clip(grads, None, loss_scale, float("inf"), None)
    return _clip(grads, None, loss_scale, float("inf"), None)


def clip_gradients(grads, max_norm: float, loss_scale: float = 1.0, out=None, stream=None):
    """(norm, out): ``norm`` as :func:`gradient_norm` gives it, and each gradient times
    min(1, max_norm / norm) / loss_scale.

    ``grads`` are fp16 or float32 CUDA tensors of any shapes without gaps in memory.  ``out`` (default: new
    float32 tensors) is a list of fp16 or float32 tensors with their shapes and strides; it may be
    ``grads`` itself.  A norm that is not finite clips nothing, so that what overflowed stays to be seen.
    """
    grads = _gradients(grads)
    if not here(grads[0].get_device(), stream):
        with on(grads[0].device, stream, *grads, *(out or ())):
            return clip_gradients(grads, max_norm, loss_scale, out)
    if out is None:
        out = [torch.empty_like(g, dtype=torch.float32, requires_grad=False) for g in grads]
    else:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out must have a tensor for each gradient")
        for i, (o, g) in enumerate(zip(out, grads)):
            if o.shape != g.shape or o.stride() != g.stride() or o.get_device() != g.get_device():
                raise ValueError(f"out[{i}] must have the shape, strides and device of grads[{i}]")
        for o in out:
            written(o)
    return _clip(grads, out, loss_scale, max_norm, None), out
