"""Values at the ends of their types' ranges in the head's losses, on the GPU against the definitions in
64 bits, with the tolerances of tests/test_gpu_head.py (check)."""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import (  # noqa: E402,F401
    D64, _built, check, gen, operands, targets, teacher, teacher_q)


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


@pytest.mark.parametrize("T", [40, 130])
@pytest.mark.parametrize("weight", [math.inf, -math.inf, math.nan])
def test_a_weight_that_is_not_finite_stays_in_its_row(T, weight):
    """The other rows' dx is what it is without that row; dW, a sum over the rows, is not finite."""
    V, D = 300, 40
    x, w = operands(T, V, D, 0, 240)
    target, (index, logits) = targets(T, V, 241, 0.0), teacher(T, V, 6, 242, torch.float16)
    index[7, 0] = 5  # row 7 has an entry
    dloss = torch.rand(T, generator=gen(243), device="cuda") + 0.5
    without, bad = dloss.clone(), dloss.clone()
    without[7], bad[7] = 0.0, weight
    rest = torch.arange(T, device="cuda") != 7
    for step in (lambda d: tg.linear_cross_entropy_step(x, w, target, d),
                 lambda d: tg.linear_distillation_step(x, w, index, logits, d)):
        loss, dx, dw = step(bad)
        want = step(without)
        assert torch.isfinite(loss).all() and torch.equal(loss, want[0])
        assert torch.equal(dx[rest], want[1][rest]) and torch.isfinite(want[1]).all()
        assert not torch.isfinite(dx[7]).any() and not torch.isfinite(dw).all()
    alone = torch.full((T,), weight, device="cuda")  # no finite weight at all
    _, dx, dw = tg.linear_cross_entropy_step(x, w, target, alone)
    assert not torch.isfinite(dx).any()
