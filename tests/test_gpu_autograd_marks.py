"""What autograd has to be told or has to refuse around the operators' kernels, which write tensors
without torch knowing."""

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402
from tests.test_gpu_head_autograd import _built, leaf  # noqa: E402,F401


def test_a_norm_over_a_saved_tensor_is_noticed():
    # relu_matmul keeps its output for the mask of its backward pass
    a, b = leaf(16, 32, seed=20), leaf(32, 64, seed=21)
    c = autograd.relu_matmul(a, b)
    with torch.no_grad():
        tg.layer_norm(c, out=c)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        c.sum().backward()
    # through a view of it too, and on another stream
    for stream in (None, torch.cuda.Stream()):
        c = autograd.relu_matmul(a, b)
        tg.layer_norm(c.detach()[:8], out=c.detach()[:8], stream=stream)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            c.sum().backward()
    # and in grad mode it is refused, as torch refuses out= of a tensor that requires a gradient
    c = autograd.relu_matmul(a, b)
    with pytest.raises(ValueError):
        tg.layer_norm(c, out=c)
    c.sum().backward()
    assert torch.isfinite(a.grad).all()


def test_other_outputs_are_as_before():
    x = leaf(4, 64, seed=22).detach()
    want = tg.layer_norm(x)
    out = torch.empty_like(x)
    before = out._version
    assert tg.layer_norm(x, out=out) is out and torch.equal(out, want) and out._version == before + 1
    with torch.inference_mode():
        out = torch.empty_like(x)
        assert torch.equal(tg.layer_norm(x, out=out), want)


@pytest.mark.parametrize("which", ["layer_norm", "linear_cross_entropy", "linear_distillation"])
def test_second_derivatives_are_refused(which):
    """Their backward kernels have no derivative: it must not come out as zero."""
    x, w = leaf(6, 16, seed=23), leaf(40, 16, seed=24)
    if which == "layer_norm":
        total = autograd.layer_norm(x, leaf(16, seed=25)).float().square().sum()
    elif which == "linear_cross_entropy":
        total = autograd.linear_cross_entropy(x, w, torch.arange(6, device="cuda"))
    else:
        index = torch.arange(24, device="cuda").view(6, 4)
        total = autograd.linear_distillation(x, w, index, leaf(6, 4, seed=26).detach())
    (dx,) = torch.autograd.grad(total, x, create_graph=True)
    assert torch.isfinite(dx).all()
    with pytest.raises(RuntimeError):  # a gradient penalty beside the loss
        (total + dx.float().square().sum()).backward()


def test_a_teacher_that_wants_a_gradient_is_refused():
    x, w, logits = leaf(6, 16, seed=27), leaf(40, 16, seed=28), leaf(6, 4, seed=29)
    index = torch.arange(24, device="cuda").view(6, 4)
    with pytest.raises(ValueError, match="detach"):
        autograd.linear_distillation(x, w, index, logits)
    autograd.linear_distillation(x, w, index, logits.detach()).backward()
    assert torch.isfinite(x.grad).all() and logits.grad is None
    with torch.no_grad():
        assert torch.isfinite(autograd.linear_distillation(x, w, index, logits))
