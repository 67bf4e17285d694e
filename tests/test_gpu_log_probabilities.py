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
