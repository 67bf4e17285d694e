"""Values at the ends of their types' ranges in the head's losses, on the GPU against the definitions in
64 bits, with the tolerances of tests/test_gpu_head.py (check)."""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import (  # noqa: E402,F401
    D64, _built, check, gen, operands, teacher_q, targets)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("tau", [0.25, 1.0, 4.0])
@pytest.mark.parametrize("top", [5, 200])
def test_teacher_logits_at_the_ends_of_their_type(dtype, tau, top):
    """Entries masked by the type's lowest value, rows of nothing else (a flat teacher), its largest
    value, and both at once; beside rows at -inf (no teacher)."""
    T, V, D = 12, 300, 40
    x, w = operands(T, V, D, 0, 210)
    index = torch.stack([torch.randperm(V, device="cuda", generator=gen(211 + t))[:top]
                         for t in range(T)])
    logits = (torch.randn(T, top, generator=gen(230), device="cuda") * 3).to(dtype)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    logits[0, 2:] = low
    logits[1] = low
    logits[2] = high
    logits[3, :3] = high
    logits[4, 0], logits[4, 1:] = high, low
    logits[5, 1:] = -math.inf
    logits[6, 1:], logits[6, 0] = -math.inf, low
    logits[7] = -math.inf
    index[8, 1:], logits[8] = -1, low
    dloss = torch.rand(T, generator=gen(231), device="cuda") + 0.5
    q, live, entropy = teacher_q(index, logits, tau, V)
    assert live.tolist() == [t != 7 for t in range(T)]
    loss, lse = tg.linear_distillation(x, w, index, logits, temperature=tau, return_lse=True)
    check(x, w, 0, 1 / tau, q, live, entropy, None, loss, lse, None, None)
    step = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=tau)
    check(x, w, 0, 1 / tau, q, live, entropy, dloss, step[0], None, step[1], step[2])
