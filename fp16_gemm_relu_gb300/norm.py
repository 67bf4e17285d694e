"""Layer normalisation of CUDA fp16 rows, forward and backward, over the C ABI
(tg_layernorm_f16, tg_layernorm_backward_f16).

    y = (x - mean) * rstd * gamma + beta,   rstd = 1 / sqrt(var + eps)

Statistics and sums are float32; fp16 outputs are rounded once.  ``autograd.layer_norm`` is the
differentiable form.
"""

from __future__ import annotations

import torch

from . import binding
from .tensors import check, here, library, on, param_type, ptr, rows, stream_handle, vector, written


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, stats: bool = False, out=None,
               stream=None):
    """y = layer norm of each row of ``x`` (M, N), N up to 32768, for a CUDA fp16 tensor with unit
    column stride; ``gamma`` and ``beta`` are (N,) fp16 or float32, or None for 1 and 0.

    Returns y, or with ``stats`` (y, mean, rstd), mean and rstd float32 (M,) as
    :func:`layer_norm_backward` takes them.  ``out`` may be a row-major (M, N) view, or x itself; autograd
    sees that it was written, and refuses a backward pass that needs what it held before.
    Runs on ``stream`` (default: torch's current stream) and returns without synchronising.
    """
    ldx = rows(x, "x")
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, x, gamma, beta, out):
            return layer_norm(x, gamma, beta, eps, stats, out)
    M, N = x.shape
    kind = binding.TG_TYPE_F16
    if gamma is not None:
        kind = param_type(gamma, "gamma")
        vector(gamma, N, dev, "gamma")
    if beta is not None:
        kind = param_type(beta, "beta")
        vector(beta, N, dev, "beta")
        if gamma is not None and gamma.dtype is not beta.dtype:
            raise TypeError("gamma and beta must have one type")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
        ldy = N
    else:
        if out.shape != x.shape or out.get_device() != dev:
            raise ValueError("out must be an (M, N) tensor on x's device")
        ldy = rows(out, "out")
        written(out)
    mean = rstd = None
    if stats:
        mean = torch.empty(M, dtype=torch.float32, device=x.device)
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    check(library().tg_layernorm_f16(x.data_ptr(), ptr(gamma), ptr(beta), out.data_ptr(), ptr(mean),
                                     ptr(rstd), M, N, ldx, ldy, eps, kind,
                                     stream_handle(dev)), "tg_layernorm_f16")
    return (out, mean, rstd) if stats else out


def layer_norm_backward(dy, x, mean, rstd, gamma=None, param_grads: bool = True, stream=None):
    """(dx, dgamma, dbeta) of :func:`layer_norm` for the upstream gradient ``dy`` (M, N) fp16.

    dgamma and dbeta have gamma's type (float32 without a gamma); with ``param_grads=False`` they
    are None and not computed.
    """
    lddy, ldx = rows(dy, "dy"), rows(x, "x")
    dev = x.get_device()
    if not here(dev, stream):
        with on(x.device, stream, dy, x, mean, rstd, gamma):
            return layer_norm_backward(dy, x, mean, rstd, gamma, param_grads)
    M, N = x.shape
    if dy.shape != x.shape or dy.get_device() != dev:
        raise ValueError("dy must have x's shape and device")
    vector(mean, M, dev, "mean")
    vector(rstd, M, dev, "rstd")
    if mean.dtype is not torch.float32 or rstd.dtype is not torch.float32:
        raise TypeError("mean and rstd must be torch.float32")
    kind, dtype = binding.TG_TYPE_F32, torch.float32
    if gamma is not None:
        kind, dtype = param_type(gamma, "gamma"), gamma.dtype
        vector(gamma, N, dev, "gamma")
    device = x.device
    dx = torch.empty((M, N), dtype=torch.float16, device=device)
    dgamma = dbeta = None
    if param_grads:
        dgamma = torch.empty(N, dtype=dtype, device=device)
        dbeta = torch.empty(N, dtype=dtype, device=device)
    check(library().tg_layernorm_backward_f16(
        dy.data_ptr(), x.data_ptr(), ptr(gamma), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
        ptr(dgamma), ptr(dbeta), M, N, lddy, ldx, N, kind, stream_handle(dev)),
        "tg_layernorm_backward_f16")
    return dx, dgamma, dbeta
