"""Log probabilities of the preference and policy losses: against themselves, as a reference; and where their sums
are exact, or a target is certain.

What the tensor cores cut off a logit's sums is put back as it is for sums of many terms of any size: of a sum v of
n <= 48 instructions (0.266 n + 0.38) 2^-24 |v| and up to 0.035 n 2^-24 |v| more, at most 8.9e-7 |v|.  Where nothing
was cut off, that is how far off the logit is, with a rounding of 2^-24 for each of the segments' additions.
"""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import D64, _built, gen  # noqa: E402,F401

PUT_BACK = (0.266 * 48 + 0.38 + 0.035 * 48) * 2 ** -24


def example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("tune_preference",
                                                  os.path.join(root, "examples", "tune_preference.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("T,V,D,layout", [
    (2048, 8192, 2048, tg.TG_HEAD_VOCAB_MAJOR), (1000, 7033, 1596, tg.TG_HEAD_VOCAB_MAJOR),
    (1024, 2501, 1024, tg.TG_HEAD_WIDTH_MAJOR), (48, 30666, 768, tg.TG_HEAD_VOCAB_MAJOR)])
def test_an_unmoved_model_has_no_margin(T, V, D, layout):
    """Against its own log probabilities a model's ratios are 0 but for the roundings of a token's: of a logit below 8
    and of the sum's logarithm below 16, 2^-22 + 2^-21 < 2^-20 at worst, which do not lean; n 2^-21 allows for half of
    them to point in one direction.  (Minus linear_cross_entropy as the reference: 3.5e-6 to 4.6e-6, 7 to 10 times
    that, a token at these sizes.)"""
    g = gen(1)
    x = torch.randn(T, D, generator=g, device="cuda").half()
    w = (torch.randn(V, D, generator=g, device="cuda") * (2 / math.sqrt(D))).half()
    if layout == tg.TG_HEAD_WIDTH_MAJOR:
        w = w.t().contiguous()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::7] = -100
    zero = torch.zeros(T, device="cuda")
    reference = tg.linear_policy(x, w, target, zero, zero, layout=layout)[1]
    assert (reference[::7] == 0).all()
    offsets = torch.tensor([0, T // 8, T], device="cuda")
    count = torch.tensor([int((target[:T // 8] >= 0).sum()), int((target[T // 8:] >= 0).sum())], device="cuda")
    one = torch.ones(1, device="cuda")
    for _, ratios, *_ in (tg.linear_preference(x, w, target, offsets, reference, layout=layout),
                          tg.linear_preference_step(x, w, target, offsets, one, reference, layout=layout),
                          tg.linear_preference_step(x, w, target, offsets, one, reference, layout=layout,
                                                    piece_rows=T // 3)):
        assert (ratios[0].abs() <= count * 2 ** -21).all(), ratios


def test_the_examples_reference():
    """tune_preference.py's reference is its own model's log probabilities: no margin before the first step, for
    answers of any lengths."""
    mod = example()
    T, D, V = 1024, 1024, 4000
    g = gen(2)

    def normal(*shape, size):
        return (torch.randn(*shape, generator=g, device="cuda") * size).half()

    w = {"gate": normal(D, D, size=D ** -0.5), "up": normal(D, D, size=D ** -0.5), "down": normal(D, D, size=D ** -0.5),
         "gamma": normal(D, size=0.1) + 1, "beta": normal(D, size=0.1), "head": normal(V, D, size=2 * D ** -0.5)}
    x = normal(T, D, size=1.0)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    reference = mod.log_probabilities(x, w, target)
    offsets = torch.tensor([0, 24, T], device="cuda")
    ratios = tg.linear_preference(mod.features(x, w), w["head"], target, offsets, reference)[1][0]
    assert (ratios.abs() <= torch.tensor([24, T - 24], device="cuda") * 2 ** -21).all(), ratios


def rows_of(kind, T, V, D):
    g = gen(3)

    def integers(*shape, lo, hi):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").half()

    if kind == "one entry":
        x = torch.zeros(T, D, device="cuda").half()
        x[torch.arange(T), torch.randint(0, D, (T,), generator=g, device="cuda")] = 4.0
        return x, torch.randn(V, D, generator=g, device="cuda").half()
    if kind == "one entry a segment":
        x = torch.zeros(T, D, device="cuda").half()
        x[:, 5::768] = 1.5
        return x, torch.randn(V, D, generator=g, device="cuda").half()
    if kind == "few entries":
        x = integers(T, D, lo=-2, hi=2) * (torch.rand(T, D, generator=g, device="cuda") < 0.02)
        return x.half(), integers(V, D, lo=-15, hi=15) / 16
    return integers(T, D, lo=-2, hi=2), integers(V, D, lo=-1, hi=1) / 4


@pytest.mark.parametrize("kind", ["one entry", "one entry a segment", "few entries", "small integers"])
@pytest.mark.parametrize("T,V,D", [(3, 900, 768), (200, 1000, 1536), (600, 2049, 2000)])
def test_exact_sums(kind, T, V, D):
    """Sums of which nothing is cut off."""
    x, w = rows_of(kind, T, V, D)
    target = torch.randint(0, V, (T,), generator=gen(4), device="cuda")
    zero = torch.zeros(T, device="cuda")
    z = x.to(D64) @ w.to(D64).t()
    segments = sum((x[:, a:a + 768].to(D64) @ w[:, a:a + 768].to(D64).t()).abs() for a in range(0, D, 768))
    dz = (PUT_BACK + math.ceil(D / 768) * 2 ** -24) * segments
    at = target[:, None]
    lse, zt = torch.logsumexp(z, 1), z.gather(1, at)[:, 0]
    # the softmax's sum moves by at most the largest logit's error; scaling by log2(e) and back, exp2f, log2f, the sum
    # over the row's parts (2^-21 of it) and the subtraction
    tol = dz.gather(1, at)[:, 0] + dz.amax(1) + 2 ** -21 * (lse.abs() + zt.abs() + 1)
    want = zt - lse
    for got in (tg.linear_policy(x, w, target, zero, zero)[1],
                tg.linear_policy_step(x, w, target, zero, zero, zero)[1]):
        assert ((got.to(D64) - want).abs() <= tol).all(), float(((got.to(D64) - want).abs() / tol).max())


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("V,D", [(1, 64), (1, 2000), (500, 64), (3000, 1536)])
def test_certain_targets(T, V, D):
    """A class alone, or one that all others are far behind, has the log probability 0: nothing of its row goes
    through an exponential, and nothing is put back for that."""
    x = torch.zeros(T, D, device="cuda").half()
    x[:, 1] = 1.0
    w = torch.zeros(V, D, device="cuda").half()
    w[1:, 1] = -1000.0  # logits 0 and -1000
    target = torch.zeros(T, dtype=torch.int64, device="cuda")
    zero = torch.zeros(T, device="cuda")
    for got in (tg.linear_policy(x, w, target, zero, zero)[1],
                tg.linear_policy_step(x, w, target, zero, zero, zero)[1]):
        assert (got == 0).all(), got
    offsets = torch.tensor([0, 1, T], device="cuda")
    assert (tg.linear_preference(x, w, target, offsets)[1] == 0).all()
