"""Losses of a linear head over a large vocabulary, with their gradients, over the C ABI
(tg_linear_cross_entropy_f16, tg_linear_distill_f16).  A cross entropy alone keeps no logits.  A step,
and distillation from a (D, V) weight, keep those of a piece of the tokens in the library's scratch: all
of them up to 2^29 (float32, and with a gradient half as much again: 3 GB) unless ``piece_rows`` is less.

``x`` is (T, D) fp16; ``weight`` is (V, D) fp16, or (D, V) with ``layout=TG_HEAD_WIDTH_MAJOR``;
losses and the log of the softmax's sum are float32 (T,).  The ``*_step`` functions compute the loss
and the gradients of sum_t dloss[t] * loss[t] in one call (three products); the others the loss
alone.  ``autograd.linear_cross_entropy`` and ``autograd.linear_distillation`` are the
differentiable forms.  All run on ``stream`` (default: torch's current stream) and return without
synchronising.
"""

from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import TG_HEAD_VOCAB_MAJOR
from .tensors import check, here, library, on, param_type, ptr, rows, stream_handle, vector

_LAYOUTS = {}


def _options(layout, piece_rows):
    """The options block: one kept per layout without other options."""
    if piece_rows == 0 and layout in _LAYOUTS:
        return _LAYOUTS[layout]
    o = ctypes.pointer(binding.tg_head_options(layout=int(layout), piece_rows=int(piece_rows)))
    if piece_rows == 0:
        _LAYOUTS[layout] = o
    return o


def _sizes(x, weight, layout):
    if layout not in (binding.TG_HEAD_VOCAB_MAJOR, binding.TG_HEAD_WIDTH_MAJOR):
        raise ValueError("layout must be TG_HEAD_VOCAB_MAJOR or TG_HEAD_WIDTH_MAJOR")
    ldx, ldw = rows(x, "x"), rows(weight, "weight")
    T, D = x.shape
    V, wd = weight.shape if layout == TG_HEAD_VOCAB_MAJOR else weight.shape[::-1]
    if wd != D:
        raise ValueError(f"x has width {D}, weight {wd}")
    if weight.get_device() != x.get_device():
        raise ValueError("weight must be on x's device")
    return T, V, D, ldx, ldw


def _teacher(index, logits, T, dev):
    if index.dtype != torch.int64:
        raise TypeError("teacher_index must be torch.int64")
    kind = param_type(logits, "teacher_logits")
    if index.dim() != 2 or index.shape[0] != T or logits.shape != index.shape:
        raise ValueError(f"teacher_index and teacher_logits must be ({T}, top)")
    if index.get_device() != dev or logits.get_device() != dev:
        raise ValueError("the teacher's entries must be on x's device")
    top = index.shape[1]
    if not 1 <= top <= binding.TG_HEAD_MAX_TOP:
        raise ValueError(f"a row has 1 to {binding.TG_HEAD_MAX_TOP} teacher entries, got {top}")
    if not index.is_contiguous() or not logits.is_contiguous():
        raise ValueError("teacher_index and teacher_logits must be contiguous")
    return top, kind


def _outputs(x, weight, T, D, need_dx, need_dw, want_lse):
    dev = x.device
    return (torch.empty(T, dtype=torch.float32, device=dev),
            torch.empty(T, dtype=torch.float32, device=dev) if want_lse else None,
            torch.empty((T, D), dtype=torch.float16, device=dev) if need_dx else None,
            torch.empty(weight.shape, dtype=torch.float16, device=dev) if need_dw else None)


def _weights(dloss, T, dev):
    if dloss is not None:
        if dloss.dtype is not torch.float32:
            raise TypeError("dloss must be torch.float32")
        vector(dloss, T, dev, "dloss")


def _cross_entropy(x, weight, target, dloss, need_dx, need_dw, want_lse, ignore_index, logit_scale,
                   layout, piece_rows, stream):
    """(loss, lse, dx, dweight), None for what is not wanted."""
    T, V, D, ldx, ldw = _sizes(x, weight, layout)
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, x, weight, target, dloss):
            return _cross_entropy(x, weight, target, dloss, need_dx, need_dw, want_lse,
                                  ignore_index, logit_scale, layout, piece_rows, None)
    if target.dtype is not torch.int64:
        raise TypeError("target must be torch.int64")
    vector(target, T, dev, "target")
    _weights(dloss, T, dev)
    out = _outputs(x, weight, T, D, need_dx, need_dw, want_lse)
    loss, lse, dx, dw = out
    check(library().tg_linear_cross_entropy_f16(
        x.data_ptr(), weight.data_ptr(), target.data_ptr(), ignore_index, logit_scale, ptr(dloss),
        loss.data_ptr(), ptr(lse), ptr(dx), ptr(dw), T, V, D, ldx, ldw, D, weight.shape[1],
        _options(layout, piece_rows), stream_handle(dev)), "tg_linear_cross_entropy_f16")
    return out


def _distillation(x, weight, teacher_index, teacher_logits, dloss, need_dx, need_dw, want_lse,
                  temperature, layout, piece_rows, stream):
    """(loss, lse, dx, dweight), None for what is not wanted."""
    T, V, D, ldx, ldw = _sizes(x, weight, layout)
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, x, weight, teacher_index, teacher_logits, dloss):
            return _distillation(x, weight, teacher_index, teacher_logits, dloss, need_dx, need_dw,
                                 want_lse, temperature, layout, piece_rows, None)
    top, kind = _teacher(teacher_index, teacher_logits, T, dev)
    _weights(dloss, T, dev)
    out = _outputs(x, weight, T, D, need_dx, need_dw, want_lse)
    loss, lse, dx, dw = out
    check(library().tg_linear_distill_f16(
        x.data_ptr(), weight.data_ptr(), teacher_index.data_ptr(), teacher_logits.data_ptr(), kind,
        top, top, temperature, ptr(dloss), loss.data_ptr(), ptr(lse), ptr(dx), ptr(dw), T, V, D,
        ldx, ldw, D, weight.shape[1], _options(layout, piece_rows), stream_handle(dev)),
        "tg_linear_distill_f16")
    return out


def linear_cross_entropy(x, weight, target, ignore_index: int = -100, logit_scale: float = 1.0,
                         layout: int = TG_HEAD_VOCAB_MAJOR, return_lse: bool = False,
                         piece_rows: int = 0, stream=None):
    """loss[t] = log sum_v exp z[t, v] - z[t, target[t]], z = logit_scale * x @ weight.T.

    ``target`` is int64 (T,); rows at ``ignore_index`` have loss 0, other targets outside the
    vocabulary NaN.  Returns loss, or (loss, lse) with ``return_lse``.
    """
    loss, lse, _, _ = _cross_entropy(x, weight, target, None, False, False, return_lse,
                                     ignore_index, logit_scale, layout, piece_rows, stream)
    return (loss, lse) if return_lse else loss


def linear_cross_entropy_step(x, weight, target, dloss, ignore_index: int = -100,
                              logit_scale: float = 1.0, layout: int = TG_HEAD_VOCAB_MAJOR,
                              piece_rows: int = 0, stream=None):
    """(loss, dx, dweight) of :func:`linear_cross_entropy` for the upstream gradient ``dloss``
    (float32 (T,)); dx is (T, D) and dweight has weight's layout, both fp16."""
    loss, _, dx, dw = _cross_entropy(x, weight, target, dloss, True, True, False, ignore_index,
                                     logit_scale, layout, piece_rows, stream)
    return loss, dx, dw


def linear_distillation(x, weight, teacher_index, teacher_logits, temperature: float = 1.0,
                        layout: int = TG_HEAD_VOCAB_MAJOR, return_lse: bool = False,
                        piece_rows: int = 0, stream=None):
    """loss[t] = sum_e q[t, e] (log q[t, e] - log p[t, teacher_index[t, e]]), q the softmax of a
    row's teacher entries over ``temperature`` and p that of x @ weight.T over the vocabulary.

    ``teacher_index`` is int64 (T, top), -1 where a row has fewer entries; ``teacher_logits`` is
    (T, top) fp16 or float32.  Returns loss, or (loss, lse) with ``return_lse``.
    """
    loss, lse, _, _ = _distillation(x, weight, teacher_index, teacher_logits, None, False, False,
                                    return_lse, temperature, layout, piece_rows, stream)
    return (loss, lse) if return_lse else loss


def linear_distillation_step(x, weight, teacher_index, teacher_logits, dloss,
                             temperature: float = 1.0, layout: int = TG_HEAD_VOCAB_MAJOR,
                             piece_rows: int = 0, stream=None):
    """(loss, dx, dweight) of :func:`linear_distillation` for the upstream gradient ``dloss``."""
    loss, _, dx, dw = _distillation(x, weight, teacher_index, teacher_logits, dloss, True, True,
                                    False, temperature, layout, piece_rows, stream)
    return loss, dx, dw
