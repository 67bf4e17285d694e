"""relu(A·B) as a differentiable torch operation whose forward and backward both run in the
library's kernels (the practitioner page, section 3.3, wraps a hand-written kernel in
torch.autograd.Function and pairs it with hand-written backward kernels).

Forward:  C = fp16(relu(A·B))                         tg_gemm_relu_f16
Backward: dZ = C > 0 ? dC : +0                        tg_relu_backward_f16
          dA = dZ·B^T  (fp32 accumulate, fp16 out)    tg_gemm_f16_t(trans_b = 1)
          dB = A^T·dZ                                  tg_gemm_f16_t(trans_a = 1)

Likewise layer normalisation, the gated feed-forward product and the losses of a linear head: layer_norm,
gated_linear, linear_cross_entropy, linear_distillation, linear_preference and linear_policy.  The
losses' forward pass is the loss alone and their backward pass the whole
step (the logits are computed again, not kept); head.linear_cross_entropy_step and the others' steps
give loss and gradients in one call where the upstream gradient is
known beforehand, a quarter of the products fewer.  Their gradients cannot be differentiated again
(that raises).
"""

from __future__ import annotations

import functools

import torch

from . import binding, gated, head, norm
from .binding import TG_ACT_SILU, TG_HEAD_VOCAB_MAJOR


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("expected a row-major 2-D tensor")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def relu_backward(dC: torch.Tensor, C: torch.Tensor) -> torch.Tensor:
    M, N = C.shape
    dZ = torch.empty_like(C)
    s = torch.cuda.current_stream(C.device).cuda_stream
    st = binding.tg_relu_backward_f16(dC.data_ptr(), C.data_ptr(), dZ.data_ptr(), M, N,
                                      _ld(dC), _ld(C), _ld(dZ), s)
    if st != binding.TG_OK:
        raise binding.TgError(st, "tg_relu_backward_f16")
    return dZ


def gemm_t(A: torch.Tensor, B: torch.Tensor, trans_a: int, trans_b: int) -> torch.Tensor:
    """op(A)·op(B) in fp16 with fp32 accumulation (op = transpose when trans_* is 1)."""
    M = A.shape[1] if trans_a else A.shape[0]
    K = A.shape[0] if trans_a else A.shape[1]
    N = B.shape[0] if trans_b else B.shape[1]
    C = torch.empty((M, N), dtype=torch.float16, device=A.device)
    s = torch.cuda.current_stream(A.device).cuda_stream
    st = binding.tg_gemm_f16_t(trans_a, trans_b, A.data_ptr(), B.data_ptr(), C.data_ptr(), M, N,
                               K, _ld(A), _ld(B), _ld(C), binding.TG_ACT_NONE, 0, 0, 0, None, s)
    if st != binding.TG_OK:
        raise binding.TgError(st, "tg_gemm_f16_t")
    return C


class ReluMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, B):
        C = binding.gemm_relu(A, B)
        ctx.save_for_backward(A, B, C)
        return C

    @staticmethod
    def backward(ctx, dC):
        A, B, C = ctx.saved_tensors
        dC = dC.to(torch.float16).contiguous()
        dZ = relu_backward(dC, C)
        dA = gemm_t(dZ, B, 0, 1) if ctx.needs_input_grad[0] else None
        dB = gemm_t(A, dZ, 1, 0) if ctx.needs_input_grad[1] else None
        return dA, dB


def relu_matmul(A: torch.Tensor, B: torch.Tensor) -> torch.Tensor:
    """Differentiable C = relu(A·B) for CUDA fp16 tensors."""
    return ReluMatmul.apply(A, B)


class _Refusal(torch.autograd.Function):
    """Passes a gradient on; its own derivative raises."""

    @staticmethod
    def forward(ctx, marker, grad):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the gradients of this operator cannot be differentiated again")


def _once(backward):
    """For backward passes of kernels alone: under create_graph=True their results are marked, or a
    second derivative would take them for constants.  (torch's once_differentiable marks them only when
    the upstream gradient requires one, which a loss's does not.)"""
    @functools.wraps(backward)
    def run(ctx, *upstream):
        with torch.no_grad():
            grads = backward(ctx, *upstream)
        if not torch.is_grad_enabled():
            return grads
        marker = torch.empty(0, requires_grad=True)
        return tuple(None if g is None else _Refusal.apply(marker, g) for g in grads)
    return run


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps):
        y, mean, rstd = norm.layer_norm(x, gamma, beta, eps, stats=True)
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.beta_dtype = None if beta is None else beta.dtype
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        want = ctx.needs_input_grad
        dx, dgamma, dbeta = norm.layer_norm_backward(dy.to(torch.float16).contiguous(), x, mean,
                                                     rstd, gamma, param_grads=want[1] or want[2])
        if want[2] and dbeta.dtype != ctx.beta_dtype:  # a beta without a gamma
            dbeta = dbeta.to(ctx.beta_dtype)
        return (dx if want[0] else None, dgamma if want[1] else None, dbeta if want[2] else None,
                None)


def layer_norm(x: torch.Tensor, gamma=None, beta=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer normalisation of the rows of a CUDA fp16 (M, N) tensor."""
    return LayerNorm.apply(x, gamma, beta, eps)


class LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, target, ignore_index, logit_scale, layout):
        ctx.save_for_backward(x, weight, target)
        ctx.args = (ignore_index, logit_scale, layout)
        return head.linear_cross_entropy(x, weight, target, ignore_index, logit_scale, layout)

    @staticmethod
    @_once
    def backward(ctx, dloss):
        x, weight, target = ctx.saved_tensors
        want = ctx.needs_input_grad
        _, _, dx, dw = head._cross_entropy(x, weight, target, dloss.contiguous(), want[0], want[1],
                                           False, *ctx.args, 0, None)
        return dx, dw, None, None, None, None


class LinearDistillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, teacher_index, teacher_logits, temperature, layout):
        ctx.save_for_backward(x, weight, teacher_index, teacher_logits)
        ctx.args = (temperature, layout)
        return head.linear_distillation(x, weight, teacher_index, teacher_logits, temperature,
                                        layout)

    @staticmethod
    @_once
    def backward(ctx, dloss):
        x, weight, teacher_index, teacher_logits = ctx.saved_tensors
        want = ctx.needs_input_grad
        _, _, dx, dw = head._distillation(x, weight, teacher_index, teacher_logits,
                                          dloss.contiguous(), want[0], want[1], False, *ctx.args,
                                          0, None)
        return dx, dw, None, None, None, None


def _reduce(loss, count, reduction):
    if reduction == "none":
        return loss
    if reduction == "sum":
        return loss.sum()
    if reduction == "mean":
        return loss.sum() / count().clamp_min(1)
    raise ValueError("reduction must be none, sum or mean")


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean",
                         logit_scale: float = 1.0,
                         layout: int = TG_HEAD_VOCAB_MAJOR) -> torch.Tensor:
    """Differentiable cross entropy of x @ weight.T (see head.linear_cross_entropy); "mean" is over the
    rows whose target is not ignore_index."""
    loss = LinearCrossEntropy.apply(x, weight, target, ignore_index, logit_scale, layout)
    return _reduce(loss, lambda: (target != ignore_index).sum(), reduction)


def linear_distillation(x: torch.Tensor, weight: torch.Tensor, teacher_index: torch.Tensor,
                        teacher_logits: torch.Tensor, temperature: float = 1.0,
                        reduction: str = "mean",
                        layout: int = TG_HEAD_VOCAB_MAJOR) -> torch.Tensor:
    """Differentiable distillation from a teacher's top logits (see head.linear_distillation); "mean" is
    over the rows that have an entry.  Not multiplied by temperature squared.  The teacher gets no
    gradient: ``teacher_logits`` that require one are refused (detach them)."""
    if teacher_logits.requires_grad and torch.is_grad_enabled():
        raise ValueError("teacher_logits must not require a gradient: there is none (detach them)")
    loss = LinearDistillation.apply(x, weight, teacher_index, teacher_logits, temperature, layout)
    return _reduce(loss, lambda: (teacher_index >= 0).any(1).sum(), reduction)


class GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, trans_w, keep):
        if not keep or not any(ctx.needs_input_grad):
            return gated.gated_linear(x, w_gate, w_up, activation, trans_w)
        h, gate, up = gated.gated_linear(x, w_gate, w_up, activation, trans_w, keep=True)
        ctx.save_for_backward(x, w_gate, w_up, gate, up)
        ctx.args = (activation, trans_w)
        return h

    @staticmethod
    @_once
    def backward(ctx, dh):
        x, w_gate, w_up, gate, up = ctx.saved_tensors
        want = ctx.needs_input_grad
        dx, dwg, dwu = gated.gated_linear_backward(
            dh.to(torch.float16).contiguous(), x, w_gate, w_up, gate, up, *ctx.args,
            input_grad=want[0], weight_grads=want[1] or want[2])
        return dx, dwg if want[1] else None, dwu if want[2] else None, None, None, None


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                 activation: int = TG_ACT_SILU, trans_w: bool = False) -> torch.Tensor:
    """Differentiable act(x @ w_gate) * (x @ w_up) (see gated.gated_linear); keeps both pre-activations
    in fp16 for the backward pass, and neither where gradients are off."""
    # (a Function's forward pass sees the inputs' requires_grad alone)
    return GatedLinear.apply(x, w_gate, w_up, activation, trans_w, torch.is_grad_enabled())


def _constant(**tensors):
    """Inputs that get no gradient must not ask for one."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} must not require a gradient: there is none (detach it)")


class LinearPreference(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, target, offsets, reference, *args):
        ctx.save_for_backward(x, weight, target, offsets, reference)
        ctx.args = args
        loss, ratios = head._preference(x, weight, target, offsets, None, False, False, reference,
                                        *args, 0, None)[:2]
        ctx.mark_non_differentiable(ratios)
        return loss, ratios

    @staticmethod
    @_once
    def backward(ctx, dloss, _):
        x, weight, target, offsets, reference = ctx.saved_tensors
        want = ctx.needs_input_grad
        _, _, dx, dw = head._preference(x, weight, target, offsets, dloss.contiguous(), want[0], want[1],
                                        reference, *ctx.args, 0, None)
        return (dx, dw) + (None,) * (3 + len(ctx.args))


class LinearPolicy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, target, old, advantage, reference, *args):
        ctx.save_for_backward(x, weight, target, old, advantage, reference)
        ctx.args = args
        loss, logp = head._policy(x, weight, target, old, advantage, None, False, False, reference,
                                  *args, 0, None)[:2]
        ctx.mark_non_differentiable(logp)
        return loss, logp

    @staticmethod
    @_once
    def backward(ctx, dloss, _):
        x, weight, target, old, advantage, reference = ctx.saved_tensors
        want = ctx.needs_input_grad
        _, _, dx, dw = head._policy(x, weight, target, old, advantage, dloss.contiguous(), want[0],
                                    want[1], reference, *ctx.args, 0, None)
        return (dx, dw) + (None,) * (4 + len(ctx.args))


def linear_preference(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                      offsets: torch.Tensor, reference=None, beta: float = 0.1,
                      label_smoothing: float = 0.0, average: bool = False, ignore_index: int = -100,
                      reduction: str = "mean", logit_scale: float = 1.0,
                      layout: int = TG_HEAD_VOCAB_MAJOR):
    """Differentiable (loss, ratios) of pairs of sequences (see head.linear_preference); "mean" is over the
    pairs.  The ratios are for looking at: they have no gradient."""
    _constant(reference=reference)
    loss, ratios = LinearPreference.apply(x, weight, target, offsets, reference, beta, label_smoothing,
                                          average, ignore_index, logit_scale, layout)
    return _reduce(loss, lambda: torch.ones_like(loss).sum(), reduction), ratios


def linear_policy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, old: torch.Tensor,
                  advantage: torch.Tensor, reference=None, clip_low: float = 0.2,
                  clip_high: float = 0.2, kl_weight: float = 0.0, ignore_index: int = -100,
                  reduction: str = "mean", logit_scale: float = 1.0,
                  layout: int = TG_HEAD_VOCAB_MAJOR):
    """Differentiable (loss, logp) of a clipped policy (see head.linear_policy); "mean" is over the rows
    whose target is not ignore_index.  logp has no gradient."""
    _constant(old=old, advantage=advantage, reference=reference)
    loss, logp = LinearPolicy.apply(x, weight, target, old, advantage, reference, clip_low, clip_high,
                                    kl_weight, ignore_index, logit_scale, layout)
    return _reduce(loss, lambda: (target != ignore_index).sum(), reduction), logp
