"""Trains the end of a language model with this package's operators: a relu layer, a layer norm, and a
linear head over a vocabulary, against next tokens and a teacher's top logits.

    python examples/train_head.py [--steps 30] [--tokens 2048] [--width 1024] [--vocab 32000]

Everything is synthetic: a fixed random teacher reads the same inputs, its top logits are kept per
token, and the targets are its first choices.  Activations and gradients are fp16 with a loss scale;
the weights have float32 masters that plain gradient descent moves.  Prints both losses as they fall,
and what one evaluation says.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402


class Student:
    """relu(x A) -> layer norm -> head; float32 masters and the fp16 weights that the kernels read."""

    def __init__(self, width: int, hidden: int, vocab: int, gen: torch.Generator):
        def normal(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale

        self.master = {
            "A": normal(width, hidden, scale=width ** -0.5),
            "gamma": torch.ones(hidden, device="cuda"),
            "beta": torch.zeros(hidden, device="cuda"),
            "head": normal(vocab, hidden, scale=0.02),
        }
        self.refresh()

    def refresh(self):
        self.w = {k: v.half().requires_grad_(True) for k, v in self.master.items()}

    def features(self, x):
        h = autograd.relu_matmul(x, self.w["A"])
        return autograd.layer_norm(h, self.w["gamma"], self.w["beta"])

    def step(self, loss_scale: float, rate: float) -> bool:
        """Moves the masters along the gradients; False (and no move) if one overflowed fp16."""
        norm, grads = tg.clip_gradients([w.grad for w in self.w.values()], float("inf"), loss_scale)
        if not bool(torch.isfinite(norm)):
            return False
        for k, g in zip(self.w, grads):
            self.master[k] -= rate * g
        self.refresh()
        return True


def run(steps: int = 30, tokens: int = 2048, width: int = 1024, vocab: int = 32000, top: int = 16,
        temperature: float = 2.0, rate: float = 2.0, quiet: bool = False) -> list[tuple[float, float]]:
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(tokens, width, generator=gen, device="cuda").half()
    # the teacher: one wide product, its largest logits kept
    teach = (x.float() @ torch.randn(width, vocab, generator=gen, device="cuda")) * (2 * width ** -0.5)
    logits, index = teach.topk(top, dim=1)
    target = index[:, 0].contiguous()
    target[::17] = -100  # padding
    del teach
    student = Student(width, width, vocab, gen)
    loss_scale = 4096.0
    seen = []
    for i in range(steps):
        y = student.features(x)
        hard = autograd.linear_cross_entropy(y, student.w["head"], target)
        soft = autograd.linear_distillation(y, student.w["head"], index, logits,
                                            temperature=temperature)
        ((hard + temperature ** 2 * soft) * loss_scale).backward()
        if not student.step(loss_scale, rate):
            loss_scale /= 2
        seen.append((float(hard.detach()), float(soft.detach())))
        if not quiet and (i % 5 == 0 or i == steps - 1):
            print(f"step {i:3d}  cross entropy {seen[-1][0]:.4f}  distillation {seen[-1][1]:.4f}")
    with torch.no_grad():  # one token's score, as when answering
        y = student.features(x[:1])
        loss, lse = tg.linear_cross_entropy(y, student.w["head"].detach(), index[:1, 0].contiguous(),
                                            return_lse=True)
    if not quiet:
        print(f"first token: loss {float(loss[0]):.4f}, log sum {float(lse[0]):.4f}")
    return seen


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    run(a.steps, a.tokens, a.width, a.vocab)


if __name__ == "__main__":
    main()
