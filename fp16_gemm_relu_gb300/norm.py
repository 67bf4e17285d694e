"""Layer normalisation of CUDA fp16 rows, forward and backward, over the C ABI
(tg_layernorm_f16, tg_layernorm_backward_f16).

    y = (x - mean) * rstd * gamma + beta,   rstd = 1 / sqrt(var + eps)

Statistics and sums are float32; fp16 outputs are rounded once.  ``autograd.layer_norm`` is the
differentiable form.
"""

from __future__ import annotations

import torch

from . import binding
from .tensors import call, param_type, rows, stream_of


def _params(gamma, beta, n, device):
    kind = binding.TG_TYPE_F16
    for p, name in ((gamma, "gamma"), (beta, "beta")):
        if p is None:
            continue
        if p.shape != (n,) or not p.is_contiguous() or p.device != device:
            raise ValueError(f"{name} must be a contiguous ({n},) tensor on x's device")
        kind = param_type(p, name)
    if gamma is not None and beta is not None and gamma.dtype != beta.dtype:
        raise TypeError("gamma and beta must have one type")
    return kind


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, stats: bool = False, out=None,
               stream=None):
    """y = layer norm of each row of ``x`` (M, N), N up to 32768, for a CUDA fp16 tensor with unit
    column stride; ``gamma`` and ``beta`` are (N,) fp16 or float32, or None for 1 and 0.

    Returns y, or with ``stats`` (y, mean, rstd), mean and rstd float32 (M,) as
    :func:`layer_norm_backward` takes them.  ``out`` may be a row-major (M, N) view, or x itself.
    Runs on ``stream`` (default: torch's current stream) and returns without synchronising.
    """
    ldx = rows(x, "x")
    M, N = x.shape
    kind = _params(gamma, beta, N, x.device)
    with stream_of(x.device, stream, x, gamma, beta, out) as handle:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float16, device=x.device)
            ldy = N
        else:
            if out.shape != x.shape or out.device != x.device:
                raise ValueError("out must be an (M, N) tensor on x's device")
            ldy = rows(out, "out")
        mean = rstd = None
        if stats:
            mean, rstd = torch.empty((2, M), dtype=torch.float32, device=x.device).unbind(0)
        call("tg_layernorm_f16", x, gamma, beta, out, mean, rstd, M, N, ldx, ldy, eps, kind, handle)
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy, x, mean, rstd, gamma=None, param_grads: bool = True, stream=None):
    """(dx, dgamma, dbeta) of :func:`layer_norm` for the upstream gradient ``dy`` (M, N) fp16.

    dgamma and dbeta have gamma's type (float32 without a gamma); with ``param_grads=False`` they
    are None and not computed.
    """
    lddy, ldx = rows(dy, "dy"), rows(x, "x")
    M, N = x.shape
    if dy.shape != x.shape or dy.device != x.device:
        raise ValueError("dy must have x's shape and device")
    for s, name in ((mean, "mean"), (rstd, "rstd")):
        if s.shape != (M,) or s.dtype != torch.float32 or s.device != x.device or (
                M > 1 and s.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous float32 (M,) tensor on x's device")
    kind = _params(gamma, None, N, x.device) if gamma is not None else binding.TG_TYPE_F32
    with stream_of(x.device, stream, dy, x, mean, rstd, gamma) as handle:
        dx = torch.empty((M, N), dtype=torch.float16, device=x.device)
        dgamma = dbeta = None
        if param_grads:
            dtype = torch.float32 if gamma is None else gamma.dtype
            dgamma = torch.empty(N, dtype=dtype, device=x.device)
            dbeta = torch.empty(N, dtype=dtype, device=x.device)
        call("tg_layernorm_backward_f16", dy, x, gamma, mean, rstd, dx, dgamma, dbeta, M, N, lddy,
             ldx, max(N, 1), kind, handle)
    return dx, dgamma, dbeta
