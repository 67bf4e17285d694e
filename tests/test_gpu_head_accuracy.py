"""How accurate the head's losses and gradients are over large vocabularies, wide rows and long batches,
as root mean squares against the definitions in 64 bits.  (tests/test_gpu_head.py holds every element to
worst-case bounds, which a systematic error could hide in.)"""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import D64, _built, gen, operands  # noqa: E402,F401


def text_targets(T, V, seed):
    """A text's tokens: frequent ones have low numbers."""
    u = torch.rand(T, generator=gen(seed), device="cuda")
    return (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)


def entries(T, V, top, seed):
    """Entries of different tokens and their logits, as float32."""
    span = V // top
    at = (torch.rand(T, top, generator=gen(seed), device="cuda") * span).long().clamp_(0, span - 1)
    index = torch.arange(top, device="cuda")[None, :] * span + at
    return index, torch.randn(T, top, generator=gen(seed + 1), device="cuda") * 3 + 10


def q_of(V, target=None, index=None, logits=None):
    """Rows of target distributions from one (T,) target or (T, top) entries, in 64 bits."""
    if target is not None:
        index, weight = target[:, None], torch.ones_like(target[:, None], dtype=D64)
    else:
        weight = torch.softmax(logits.to(D64), 1)
    return torch.zeros(index.shape[0], V, dtype=D64, device="cuda").scatter_add_(1, index, weight)


def shrink(got, ref):
    """How far `got` is from `ref` along ref itself, relative: what rounding leaves near 0."""
    return float((got.to(D64) * ref).sum() / (ref * ref).sum()) - 1


# A sum of 16384 products by the tensor core is 1024 instructions, each of which cuts off half a unit on
# average where rounding would cut off none: at most 1024 2^-24 of a sum that has its size from the start.
MOST_SHRINK = 2 ** -14


@pytest.mark.parametrize("T,V,D", [(4864, 65536, 1024), (2432, 120000, 2048), (64, 131072, 4096)])
@pytest.mark.parametrize("which", ["loss", "distil"])
def test_long_sums_over_the_vocabulary_do_not_shrink(T, V, D, which):
    x, w = operands(T, V, D, tg.TG_HEAD_VOCAB_MAJOR, 200)
    dloss = torch.full((T,), 8.0, device="cuda")
    n = 64
    if which == "loss":
        target = text_targets(T, V, 201)
        _, dx, _ = tg.linear_cross_entropy_step(x, w, target, dloss)
        q = q_of(V, target=target[:n])
    else:
        index, logits = entries(T, V, 16, 202)
        _, dx, _ = tg.linear_distillation_step(x, w, index, logits, dloss)
        q = q_of(V, index=index[:n], logits=logits[:n])
    wd = w.to(D64)
    ref = 8.0 * (torch.softmax(x[:n].to(D64) @ wd.t(), 1) - q) @ wd
    assert abs(shrink(dx[:n], ref)) <= MOST_SHRINK


def test_long_sums_over_the_tokens_do_not_shrink():
    # every token has the same target and the features are positive: the target's row of dW only grows
    T, V, D = 100000, 4864, 1024
    x, w = operands(T, V, D, tg.TG_HEAD_VOCAB_MAJOR, 204)
    x = x.abs().contiguous()
    target = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    dloss = torch.full((T,), 0.125, device="cuda")
    _, _, dw = tg.linear_cross_entropy_step(x, w, target, dloss)
    wd, ref = w.to(D64), torch.zeros(D, dtype=D64, device="cuda")
    for a in range(0, T, 10000):
        xd = x[a:a + 10000].to(D64)
        ref += 0.125 * (torch.softmax(xd @ wd.t(), 1)[:, 77] - 1) @ xd
    assert abs(shrink(dw[77], ref)) <= MOST_SHRINK
