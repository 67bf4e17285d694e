"""What autograd.gated_linear asks of its kernels, on the CPU with plain functions in their place: whether the
pre-activations are kept, and that a forward-mode derivative is refused as by the other operators."""

import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad  # noqa: E402

from fp16_gemm_relu_gb300 import autograd, gated  # noqa: E402


@pytest.fixture
def kept(monkeypatch):
    """The `keep` of each forward call."""
    seen = []

    def forward(x, w_gate, w_up, activation, trans_w=False, keep=False):
        seen.append(keep)
        g, u = x @ w_gate, x @ w_up
        h = g * u
        return (h, g, u) if keep else h

    monkeypatch.setattr(gated, "gated_linear", forward)
    return seen


def operands(requires_grad):
    return [torch.ones(s, dtype=torch.float64).requires_grad_(requires_grad) for s in ((2, 3), (3, 4), (3, 4))]


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_without_gradients(kept, off):
    with off():
        h = autograd.gated_linear(*operands(True))
    assert kept == [False] and not h.requires_grad
    assert not autograd.gated_linear(*operands(False)).requires_grad and kept == [False, False]


def test_pre_activations_are_kept_for_a_gradient(kept):
    assert autograd.gated_linear(*operands(True)).requires_grad and kept == [True]
    x, wg, wu = operands(False)
    assert autograd.gated_linear(x, wg, wu.requires_grad_(True)).requires_grad and kept == [True, True]


@pytest.mark.parametrize("on", [torch.enable_grad, torch.no_grad])
def test_forward_mode_is_refused(kept, on):
    """A tangent lives on where gradients are off: it must not be lost."""
    x, wg, wu = operands(False)
    with forward_ad.dual_level(), on():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="jvp"):
            autograd.gated_linear(dual, wg, wu)
