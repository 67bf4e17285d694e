"""Steps of few tokens over a large head, whose two gradients run side by side: captured they give the
same bits as called, at widths around the tiles', with rows that are copied first too."""

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import (  # noqa: E402,F401
    D64, _built, check, gen, one_hot, operands, targets, teacher)


@pytest.mark.parametrize("T,V,D,pad,offset", [
    (1, 28672, 1024, 0, 0), (9, 26000, 520, 0, 0), (16, 8192, 4096, 0, 0), (64, 25001, 600, 0, 0),
    (65, 13000, 1000, 0, 0), (128, 6200, 2056, 0, 0), (20, 1000, 20000, 0, 0),
    (5, 20001, 701, 0, 0), (100, 14000, 1023, 3, 1)])
@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
def test_captured_and_called(T, V, D, pad, offset, layout):
    x, w = operands(T, V, D, layout, 250, pad=pad, offset=offset)
    target, (index, logits) = targets(T, V, 251, 0.1), teacher(T, V, 9, 252, torch.float16)
    dloss = torch.rand(T, generator=gen(253), device="cuda") + 0.5
    steps = {
        "loss": lambda: tg.linear_cross_entropy_step(x, w, target, dloss, layout=layout),
        "distil": lambda: tg.linear_distillation_step(x, w, index, logits, dloss, layout=layout)}
    for which, step in steps.items():
        called = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(called, captured))
        if which == "loss":
            q, live = one_hot(target, V)
            zero = torch.zeros(T, dtype=D64, device="cuda")
            check(x, w, layout, 1.0, q, live, zero, dloss, called[0], None, *called[1:])
