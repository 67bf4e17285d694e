"""The differentiable forms of layer norm and of the head's losses, and the example that trains with
them.

Tolerances: the autograd forms call the kernels that tests/test_gpu_norm.py and tests/test_gpu_head.py
hold to 64-bit references, so here a gradient is within 2^-8 of its size or of 2^-9 of the largest of
its tensor: two fp16 roundings (2^-11 each) along the way, and their sums' partial cancellation.
"""

import importlib.util
import os

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp16_gemm_relu_gb300 import build

    build.build()
    binding.load_library()
    torch.cuda.set_device(0)
    yield
    st, word = binding.tg_device_error_check(clear=True)
    assert st == binding.TG_OK, f"device error word {word:#x}"


def leaf(*shape, seed, scale=1.0, dtype=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype).requires_grad_(True)


def near(got, want):
    want = want.to(D64)
    return bool(((got.to(D64) - want).abs() <= want.abs() * 2 ** -8 + want.abs().max() * 2 ** -9).all())


def double(*tensors):
    return [t.detach().to(D64).requires_grad_(True) for t in tensors]


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("beta_only", [False, True])
def test_layer_norm(dtype, beta_only):
    x = leaf(70, 328, seed=1)
    gamma = None if beta_only else leaf(328, seed=2, dtype=dtype)
    beta = leaf(328, seed=3, dtype=dtype)
    up = leaf(70, 328, seed=4).detach()
    y = autograd.layer_norm(x, gamma, beta)
    y.backward(up)
    xd, bd = double(x, beta)
    gd = double(gamma)[0] if gamma is not None else None
    want = torch.nn.functional.layer_norm(xd, (328,), gd, bd)
    want.backward(up.to(D64))
    assert near(y.detach(), want.detach()) and near(x.grad, xd.grad) and near(beta.grad, bd.grad)
    assert beta.grad.dtype == dtype
    if gamma is not None:
        assert gamma.grad.dtype == dtype and near(gamma.grad, gd.grad)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
def test_cross_entropy(reduction, layout):
    x, w = leaf(60, 64, seed=5), leaf(500, 64, seed=6, scale=0.2)
    if layout == tg.TG_HEAD_WIDTH_MAJOR:
        w = w.detach().t().contiguous().requires_grad_(True)
    target = torch.randint(0, 500, (60,), device="cuda")
    target[::7] = -100
    loss = autograd.linear_cross_entropy(x, w, target, reduction=reduction, layout=layout)
    xd, wd = double(x, w)
    z = xd @ (wd.t() if layout == tg.TG_HEAD_VOCAB_MAJOR else wd)
    want = torch.nn.functional.cross_entropy(z, target, reduction=reduction)
    scale = 512.0
    (loss.sum() * scale).backward()
    (want.sum() * scale).backward()
    assert torch.allclose(loss.detach().to(D64), want.detach(), rtol=1e-5, atol=1e-5)
    assert near(x.grad, xd.grad) and near(w.grad, wd.grad)


def test_distillation_of_one_operand_alone():
    x, w = leaf(40, 48, seed=7), leaf(300, 48, seed=8, scale=0.2)
    index = torch.stack([torch.randperm(300, device="cuda")[:6] for _ in range(40)])
    logits = torch.randn(40, 6, device="cuda") * 2
    xd, wd = double(x, w)
    logp = torch.log_softmax(xd @ wd.t() / 2, 1)
    q = torch.softmax(logits.to(D64) / 2, 1)
    want = (q * (q.log() - logp.gather(1, index))).sum(1).mean()
    (want * 512).backward()
    for which in ("x", "w"):
        a = x.detach().clone().requires_grad_(which == "x")
        b = w.detach().clone().requires_grad_(which == "w")
        loss = autograd.linear_distillation(a, b, index, logits, temperature=2.0)
        (loss * 512).backward()
        assert abs(float(loss.detach()) - float(want.detach())) < 1e-5 * (1 + abs(float(want.detach())))
        if which == "x":
            assert b.grad is None and near(a.grad, xd.grad)
        else:
            assert a.grad is None and near(b.grad, wd.grad)


def test_unknown_reduction():
    x, w = leaf(4, 8, seed=9), leaf(10, 8, seed=10)
    with pytest.raises(ValueError):
        autograd.linear_cross_entropy(x, w, torch.zeros(4, dtype=torch.int64, device="cuda"),
                                      reduction="median")


def test_the_example_learns():
    spec = importlib.util.spec_from_file_location("train_head",
                                                  os.path.join(ROOT, "examples", "train_head.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    seen = example.run(steps=12, tokens=512, width=256, vocab=2000, quiet=True)
    assert all(h == h and s == s for h, s in seen)
    # both losses start near those of a flat guess and fall by a tenth at least
    assert seen[-1][0] < 0.9 * seen[0][0] and seen[-1][1] < 0.9 * seen[0][1]
