"""Gradients unscaled and clipped by their global norm, over the C ABI (tg_clip_gradients).

Squares are summed in float32 by blocks, the blocks' sums in float64; results are the same run to run.
Calls run on ``stream`` (default: torch's current stream) and return without synchronising: the norm
stays on the device.
"""

from __future__ import annotations

import array

import torch

from . import binding
from .tensors import check, here, library, on, param_type, stream_handle, written

_KINDS = {torch.float16: binding.TG_TYPE_F16, torch.float32: binding.TG_TYPE_F32}


def _dense(t, name):
    """Whether t's values fill its memory without gaps, in any order of dimensions."""
    n = 1
    for stride, size in sorted((s, d) for s, d in zip(t.stride(), t.shape) if d != 1):
        if stride != n:
            raise ValueError(f"{name} must fill its memory without gaps or overlaps")
        n *= size


def _alike(a, b):
    """Whether two tensors of one shape have their values in the same order in memory: their strides say so but
    for those of dimensions of one element."""
    return a.stride() == b.stride() or (
        a.numel() == 0 or all(s == t for s, t, d in zip(a.stride(), b.stride(), a.shape) if d != 1))


def _call(words, n, loss_scale, max_norm, device, dev):
    norm = torch.empty((), dtype=torch.float32, device=device)
    table = array.array("Q", words)  # tg_gradient, four words each
    check(library().tg_clip_gradients(table.buffer_info()[0], n, loss_scale, max_norm,
                                      norm.data_ptr(), stream_handle(dev)), "tg_clip_gradients")
    return norm


def _kind(g, dev, i):
    """The type of the i-th gradient, which is a dense tensor on device ``dev``.  Calls on few small
    gradients are bound by this loop: what a good tensor needs is asked in one line."""
    kind = _KINDS.get(g.dtype)
    if kind is None or g.get_device() != dev or not g.is_contiguous():
        param_type(g, f"grads[{i}]")
        if g.get_device() != dev:
            raise ValueError("the gradients must be on one CUDA device")
        _dense(g, f"grads[{i}]")
    return kind


def _device(grads):
    if not grads:
        raise ValueError("no gradients")
    if not grads[0].is_cuda:
        raise ValueError("the gradients must be CUDA tensors")
    return grads[0].get_device()


def gradient_norm(grads, loss_scale: float = 1.0, stream=None):
    """The norm of all of ``grads`` together over ``loss_scale``, a float32 scalar on their device."""
    grads = list(grads)
    dev = _device(grads)
    if not here(dev, stream):
        with on(grads[0].device, stream, *grads):
            return gradient_norm(grads, loss_scale)
    words = []
    for i, g in enumerate(grads):
        words += (g.data_ptr(), 0, g.numel(), _kind(g, dev, i))
    return _call(words, len(grads), loss_scale, float("inf"), grads[0].device, dev)


def clip_gradients(grads, max_norm: float, loss_scale: float = 1.0, out=None, stream=None):
    """(norm, out): ``norm`` as :func:`gradient_norm` gives it, and each gradient times
    min(1, max_norm / norm) / loss_scale.

    ``grads`` are fp16 or float32 CUDA tensors of any shapes without gaps in memory.  ``out`` (default: new
    float32 tensors) holds fp16 or float32 tensors with their shapes and orders in memory; it may be
    ``grads`` itself.  A norm that is not finite clips nothing, so that what overflowed stays to be seen.
    """
    grads = list(grads)
    out = None if out is None else list(out)
    dev = _device(grads)
    if not here(dev, stream):
        with on(grads[0].device, stream, *grads, *(out or ())):
            return clip_gradients(grads, max_norm, loss_scale, out)
    words = []
    if out is None:
        out, like, kind32 = [], torch.empty_like, binding.TG_TYPE_F32 << 32
        for i, g in enumerate(grads):
            kind = _kind(g, dev, i)
            o = like(g, dtype=torch.float32)
            out.append(o)
            words += (g.data_ptr(), o.data_ptr(), g.numel(), kind | kind32)
    else:
        if len(out) != len(grads):
            raise ValueError("out must have a tensor for each gradient")
        for i, (g, o) in enumerate(zip(grads, out)):
            kind = _kind(g, dev, i)
            if o.shape != g.shape or o.get_device() != dev or not _alike(o, g):
                raise ValueError(f"out[{i}] must have the shape, order in memory and device of grads[{i}]")
            words += (g.data_ptr(), o.data_ptr(), g.numel(), kind | param_type(o, f"out[{i}]") << 32)
        for o in out:
            written(o)
    return _call(words, len(grads), loss_scale, max_norm, grads[0].device, dev), out
