"""The gated feed-forward product of CUDA fp16 tensors and its backward pass, over the C ABI
(tg_gated_f16, tg_gated_backward_f16).

    gate = x @ w_gate,  up = x @ w_up,  h = act(gate) * up

``x`` is (M, K); the weights are (K, N), or (N, K) with ``trans_w``; all fp16 with unit column stride.
Sums are float32 and every output is rounded once.  ``activation`` is TG_ACT_SILU, TG_ACT_GELU,
TG_ACT_GELU_TANH, TG_ACT_RELU or TG_ACT_NONE.  ``autograd.gated_linear`` is the differentiable form.
Calls run on ``stream`` (default: torch's current stream) and return without synchronising.
"""

from __future__ import annotations

import torch

from . import binding
from .binding import TG_ACT_SILU
from .tensors import check, here, library, on, ptr, rows, stream_handle, written

_DENSE = torch.contiguous_format


def _sizes(x, w_gate, w_up, trans_w):
    ldx, ldg, ldu = rows(x, "x"), rows(w_gate, "w_gate"), rows(w_up, "w_up")
    M, K = x.shape
    N, wk = w_gate.shape if trans_w else w_gate.shape[::-1]
    if wk != K:
        raise ValueError(f"x has width {K}, the weights {wk}")
    if w_up.shape != w_gate.shape:
        raise ValueError("w_gate and w_up must have one shape")
    dev = x.get_device()
    if w_gate.get_device() != dev or w_up.get_device() != dev:
        raise ValueError("the weights must be on x's device")
    return M, N, K, ldx, ldg, ldu


def _like(t, shape, dev, name):
    """The leading dimension of an (M, N) operand on x's device."""
    ld = rows(t, name)
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {tuple(shape)} tensor on x's device")
    return ld


def gated_linear(x, w_gate, w_up, activation: int = TG_ACT_SILU, trans_w: bool = False,
                 keep: bool = False, out=None, options=None, stream=None):
    """h = act(x @ w_gate) * (x @ w_up), or with ``keep`` (h, gate, up) as
    :func:`gated_linear_backward` takes them.

    ``out`` may be a row-major (M, N) view for h that overlaps no input; autograd sees that it was written.  ``options`` may
    hold plan overrides by name (block_n, split_k, pair, panel_m, max_ctas, timeout_ms).
    """
    M, N, K, ldx, ldg, ldu = _sizes(x, w_gate, w_up, trans_w)
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, x, w_gate, w_up, out):
            return gated_linear(x, w_gate, w_up, activation, trans_w, keep, out, options)
    ldh = N
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    else:
        ldh = _like(out, (M, N), dev, "out")
        written(out)
    gate = up = None
    if keep:
        gate, up = torch.empty_like(out, memory_format=_DENSE), torch.empty_like(out, memory_format=_DENSE)
    check(library().tg_gated_f16(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(),
                                 ptr(gate), ptr(up), activation, 1 if trans_w else 0, M, N, K, ldx,
                                 ldg, ldu, ldh, N, N, options and binding._opts(options), stream_handle(dev)),
          "tg_gated_f16")
    return (out, gate, up) if keep else out


def gated_linear_backward(dh, x, w_gate, w_up, gate, up, activation: int = TG_ACT_SILU,
                          trans_w: bool = False, input_grad: bool = True, weight_grads: bool = True,
                          options=None, stream=None):
    """(dx, dw_gate, dw_up) of :func:`gated_linear` for the upstream gradient ``dh`` (M, N), from the
    ``gate`` and ``up`` that it kept; the weights' gradients are stored as the weights are.  What
    ``input_grad=False`` or ``weight_grads=False`` leaves out is None and not computed."""
    M, N, K, ldx, ldg, ldu = _sizes(x, w_gate, w_up, trans_w)
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, dh, x, w_gate, w_up, gate, up):
            return gated_linear_backward(dh, x, w_gate, w_up, gate, up, activation, trans_w,
                                         input_grad, weight_grads, options)
    shape = (M, N)
    lddh, ldgate, ldup = _like(dh, shape, dev, "dh"), _like(gate, shape, dev, "gate"), _like(up, shape, dev, "up")
    dx = torch.empty_like(x, memory_format=_DENSE) if input_grad else None
    dwg = dwu = None
    if weight_grads:
        dwg = torch.empty_like(w_gate, memory_format=_DENSE)
        dwu = torch.empty_like(w_up, memory_format=_DENSE)
    ldw = w_gate.shape[1]
    check(library().tg_gated_backward_f16(
        dh.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), gate.data_ptr(),
        up.data_ptr(), ptr(dx), ptr(dwg), ptr(dwu), activation, 1 if trans_w else 0, M, N, K, lddh, ldx,
        ldg, ldu, ldgate, ldup, K, ldw, ldw, options and binding._opts(options), stream_handle(dev)),
        "tg_gated_backward_f16")
    return dx, dwg, dwu
