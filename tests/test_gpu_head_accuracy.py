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


def rms(got, ref):
    return float((got.to(D64) - ref).norm() / ref.norm())


@pytest.mark.parametrize("T,V,D", [(1, 28672, 8192), (40, 4099, 3000), (300, 9001, 8192),
                                   (200, 131072, 512), (128, 50257, 1600)])
@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
def test_losses(T, V, D, layout):
    """An lse near 10 carries a handful of float32 roundings (2^-24 each, 2.4e-7 for four); a segment of
    1024 products is 64 instructions that cut off half a unit each, of partial sums that grow from zero:
    about 2^-20 of a logit of 2, 2e-7 of the lse.  (Sums of 8192 in one piece put 4.5e-6 on a loss.)"""
    x, w = operands(T, V, D, layout, 260)
    wd = (w if layout == tg.TG_HEAD_VOCAB_MAJOR else w.t()).to(D64)
    z = x.to(D64) @ wd.t()
    want = torch.logsumexp(z, 1)
    target = text_targets(T, V, 261)
    loss, lse = tg.linear_cross_entropy(x, w, target, layout=layout, return_lse=True)
    assert rms(lse, want) <= 1e-6
    assert float((loss.to(D64) - (want - z.gather(1, target[:, None])[:, 0])).norm() / want.norm()) <= 1e-6
    index, logits = entries(T, V, 16, 262)
    loss, lse = tg.linear_distillation(x, w, index, logits, layout=layout, return_lse=True)
    q = torch.softmax(logits.to(D64), 1)
    ref = (q * (q.log() - z.gather(1, index) + want[:, None])).sum(1)
    assert rms(lse, want) <= 1e-6 and float((loss.to(D64) - ref).norm() / want.norm()) <= 1e-6


def gradients(x, w, layout, q, dloss, step=512):
    """(dX, dW) in 64 bits, the rows in steps: the matrix of logits may not fit at once."""
    wd = (w if layout == tg.TG_HEAD_VOCAB_MAJOR else w.t()).to(D64)
    dx, dw = torch.empty_like(x, dtype=D64), torch.zeros_like(wd)
    for a in range(0, x.shape[0], step):
        xd = x[a:a + step].to(D64)
        G = torch.softmax(xd @ wd.t(), 1) - q(a, a + step)
        G *= dloss[a:a + step, None].to(D64)
        dx[a:a + step] = G @ wd
        dw += G.t() @ xd
    return dx, dw if layout == tg.TG_HEAD_VOCAB_MAJOR else dw.t()


@pytest.mark.parametrize("T,V,D,layout", [
    (16, 131072, 512, tg.TG_HEAD_VOCAB_MAJOR), (64, 28672, 3000, tg.TG_HEAD_VOCAB_MAJOR),
    (64, 65537, 513, tg.TG_HEAD_WIDTH_MAJOR), (65, 65537, 512, tg.TG_HEAD_VOCAB_MAJOR),
    (300, 65537, 512, tg.TG_HEAD_WIDTH_MAJOR), (400, 131072, 256, tg.TG_HEAD_VOCAB_MAJOR),
    (300, 3000, 8192, tg.TG_HEAD_VOCAB_MAJOR),
    (4608, 131072, 64, tg.TG_HEAD_VOCAB_MAJOR)])  # two pieces by the default rule
@pytest.mark.parametrize("which", ["loss", "distil"])
def test_gradients(T, V, D, layout, which):
    """A rounding to fp16 is 2.0e-4 of numbers of any size, root mean square, and 2^-11 / sqrt(3) =
    2.8e-4 at most.  Up to 64 tokens the output's is the only one, beside what long sums lose (2^-14):
    2.2e-4.  With more, G's comes to it, which where one entry is most of a row is that row's: at most
    sqrt(2.1^2 + 2.8^2) = 3.5e-4."""
    x, w = operands(T, V, D, layout, 270)
    dloss = torch.full((T,), 64.0, device="cuda")  # so that the gradients are normal fp16 numbers
    if which == "loss":
        target = text_targets(T, V, 271)
        _, dx, dw = tg.linear_cross_entropy_step(x, w, target, dloss, layout=layout)
        ref = gradients(x, w, layout, lambda a, b: q_of(V, target=target[a:b]), dloss)
    else:
        index, logits = entries(T, V, 16, 272)
        _, dx, dw = tg.linear_distillation_step(x, w, index, logits, dloss, layout=layout)
        ref = gradients(x, w, layout, lambda a, b: q_of(V, index=index[a:b], logits=logits[a:b]),
                        dloss)
    most = 2.5e-4 if T <= 64 else 3.5e-4
    assert rms(dx, ref[0]) <= most and rms(dw, ref[1]) <= most


def test_rows_of_different_weight():
    """G's spacing is 2^-39 of the largest weight, so that a row of weight r times the largest keeps 11
    bits of every p from 2^-29 / r on: of nearly all of them here, down to r = 2^-13.  Then each row of dX
    is within its own two roundings (2^-11 each at most)."""
    T, V, D = 300, 3000, 256
    x, w = operands(T, V, D, 0, 280)
    target = text_targets(T, V, 281)
    dloss = 16384.0 * 2.0 ** (-13 * torch.rand(T, generator=gen(282), device="cuda"))
    dloss[0], dloss[1] = 16384.0, 2.0
    _, dx, _ = tg.linear_cross_entropy_step(x, w, target, dloss)
    ref, _ = gradients(x, w, 0, lambda a, b: q_of(V, target=target[a:b]), dloss)
    assert ((dx.to(D64) - ref).norm(dim=1) <= 2 ** -10 * ref.norm(dim=1)).all()
