"""Calls of the fine-tuning operators that lie at an edge of what they allow."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402
from tests.test_gpu_head import _built, gen  # noqa: E402,F401


def normal(*shape, seed, size=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * size).half()


@pytest.mark.parametrize("captured", [False, True])
def test_no_rows_without_a_gradient(captured):
    """An empty batch of preferences and of a policy, the value alone."""
    x, w = torch.empty(0, 64, dtype=torch.float16, device="cuda"), normal(100, 64, seed=1)
    target = torch.empty(0, dtype=torch.int64, device="cuda")
    offsets = torch.zeros(5, dtype=torch.int64, device="cuda")
    empty = torch.empty(0, device="cuda")

    def calls():
        return (*tg.linear_preference(x, w, target, offsets),
                *tg.linear_preference(x, w, target, offsets, empty, average=True),
                *tg.linear_preference(x, w, target, offsets[:1]),
                *tg.linear_policy(x, w, target, empty, empty))

    if captured:
        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls()
        for t in got:
            t.fill_(7.0)
        graph.replay()
    else:
        got = calls()
    for loss, ratios in (got[0:2], got[2:4]):
        assert ((loss - math.log(2)).abs() < 1e-6).all() and loss.shape == (2,) and (ratios == 0).all()
    assert got[4].shape == (0,) and got[5].shape == (0, 2) and got[6].shape == got[7].shape == (0,)
    loss, _ = autograd.linear_preference(x.clone().requires_grad_(True), w, target, offsets)
    assert abs(float(loss.detach()) - math.log(2)) < 1e-6
    loss.backward()
