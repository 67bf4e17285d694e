"""Tunes a small model on preferences with this package's operators: a gated block with its residual, a layer
norm and a head, the preference loss of pairs of answers against a reference (the model as it was), and
gradients unscaled and clipped by their norm.

    python examples/tune_preference.py [--steps 30] [--pairs 16] [--length 64] [--width 512] [--vocab 8000]

Everything is synthetic: random tokens of random answers, half of them called better.  Activations and
gradients are fp16 with a loss scale; the weights have float32 masters that plain gradient descent moves.
Prints the loss and how many pairs are in the right order.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402


class Project(torch.autograd.Function):
    """h @ w and its gradients through the framework's GEMMs."""

    @staticmethod
    def forward(ctx, h, w):
        ctx.save_for_backward(h, w)
        return tg.gemm_relu(h, w, epilogue=tg.TG_EPILOGUE_NONE)

    @staticmethod
    def backward(ctx, d):
        h, w = ctx.saved_tensors
        return autograd.gemm_t(d, w, 0, 1), autograd.gemm_t(h, d, 1, 0)


def features(x, w):
    h = autograd.gated_linear(x, w["gate"], w["up"])
    return autograd.layer_norm(x + Project.apply(h, w["down"]), w["gamma"], w["beta"])


def log_probabilities(x, w, target):
    """The targets' log probabilities as the preference loss has them, without a gradient."""
    with torch.no_grad():
        zero = torch.zeros(target.shape, device=target.device)  # (a policy's loss is not wanted)
        return tg.linear_policy(features(x, w), w["head"], target, zero, zero)[1]


def run(steps: int = 30, pairs: int = 16, length: int = 64, width: int = 512, hidden: int = 1024,
        vocab: int = 8000, beta: float = 0.1, rate: float = 0.5, max_norm: float = 1.0,
        quiet: bool = False) -> list[tuple[float, float]]:
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, size):
        return torch.randn(*shape, generator=gen, device="cuda") * size

    master = {"gate": normal(width, hidden, size=width ** -0.5), "up": normal(width, hidden, size=width ** -0.5),
              "down": normal(hidden, width, size=hidden ** -0.5), "gamma": torch.ones(width, device="cuda"),
              "beta": torch.zeros(width, device="cuda"), "head": normal(vocab, width, size=width ** -0.5)}
    tokens = 2 * pairs * length
    x = normal(tokens, width, size=1.0).half()
    target = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    target.view(-1, length)[:, :length // 4] = -100  # the prompts
    offsets = torch.arange(2 * pairs + 1, device="cuda") * length
    loss_scale = 4096.0
    w = {k: v.half().requires_grad_(True) for k, v in master.items()}
    reference = log_probabilities(x, w, target)  # once
    seen = []
    for i in range(steps):
        loss, ratios = autograd.linear_preference(features(x, w), w["head"], target, offsets, reference,
                                                  beta=beta)
        (loss * loss_scale).backward()
        norm, grads = tg.clip_gradients([p.grad for p in w.values()], max_norm, loss_scale)
        if bool(torch.isfinite(norm)):
            for k, g in zip(master, grads):
                master[k] -= rate * g
        else:  # a gradient overflowed fp16
            loss_scale /= 2
        w = {k: v.half().requires_grad_(True) for k, v in master.items()}
        seen.append((float(loss.detach()), float((ratios[:, 0] > ratios[:, 1]).float().mean())))
        if not quiet and (i % 5 == 0 or i == steps - 1):
            print(f"step {i:3d}  loss {seen[-1][0]:.4f}  in order {seen[-1][1]:.2f}  norm {float(norm):.3f}")
    return seen


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("steps", 30), ("pairs", 16), ("length", 64), ("width", 512), ("vocab", 8000)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    run(a.steps, a.pairs, a.length, a.width, 2 * a.width, a.vocab)


if __name__ == "__main__":
    main()
