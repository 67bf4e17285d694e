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


@pytest.mark.parametrize("piece_rows", [0, 2])
def test_a_ratio_beyond_float32_without_an_advantage(piece_rows):
    """r A is 0 for an advantage of 0, however large r is; a log probability that is NaN stays one."""
    x, w = normal(5, 64, seed=2), normal(40, 64, seed=3)
    target = torch.zeros(5, dtype=torch.int64, device="cuda")
    old = torch.tensor([-200.0, -math.inf, -200.0, math.nan, -3.0], device="cuda")
    advantage = torch.tensor([0.0, -0.0, 1.0, 0.0, 0.0], device="cuda")
    one = torch.ones(5, device="cuda")
    for kl in (0.0, 0.5):
        args = dict(reference=torch.zeros(5, device="cuda"), kl_weight=kl)
        value = tg.linear_policy(x, w, target, old, advantage, piece_rows=piece_rows, **args)
        loss, logp, dx, dw = tg.linear_policy_step(x, w, target, old, advantage, one, piece_rows=piece_rows, **args)
        d = -logp
        want = kl * (torch.expm1(d) - d)
        want[2] -= 1.2  # clipped: no gradient of its own
        good = torch.tensor([0, 1, 2, 4], device="cuda")
        for got in (loss, value[0]):
            assert got[3].isnan() and torch.allclose(got[good], want[good], rtol=1e-5, atol=1e-6)
        # (the penalty's slope is 0.5 (1 - e^d) with d up to 30 here, far beyond fp16: infinite, not NaN)
        assert dx[3].isnan().all() and not dx[good].isnan().any() and dw.isnan().any()
        if kl == 0:
            assert (dx[good] == 0).all()


def test_a_policy_clipped_from_below_alone():
    """A clip_high that no ratio reaches clips nothing."""
    x, w = normal(6, 64, seed=4), normal(40, 64, seed=5)
    target = torch.arange(6, device="cuda")
    zero = torch.zeros(6, device="cuda")
    logp = tg.linear_policy(x, w, target, zero, zero)[1]
    advantage = torch.tensor([1.0, 1.0, 1.0, -1.0, -1.0, -1.0], device="cuda")
    moved = torch.tensor([4.0, 0.0, -4.0] * 2, device="cuda")
    ratio = torch.exp(moved)
    loss, _ = tg.linear_policy(x, w, target, logp - moved, advantage, clip_high=1e30)
    want = -torch.minimum(ratio * advantage, ratio.clamp_min(0.8) * advantage)
    # old is rounded by up to 2^-20 (of values below 16), and e^m by 2^-20 of itself
    assert ((loss - want).abs() <= 2 ** -18 * want.abs()).all()


@pytest.mark.parametrize("stream", [False, True])
def test_clip_takes_any_iterable(stream):
    grads = [normal(33, 5, seed=6), normal(7, seed=7).float()]
    want = tg.clip_gradients(grads, 0.5)
    torch.cuda.synchronize()
    out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    s = torch.cuda.Stream() if stream else None
    norm, got = tg.clip_gradients(iter(grads), 0.5, out=iter(out), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(norm, want[0]) and all(a is b for a, b in zip(got, out))
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    assert torch.equal(tg.gradient_norm(iter(grads), stream=s), norm)


def test_clip_into_the_same_memory_order_under_other_strides():
    """The stride of a dimension of one element says nothing about where values lie."""
    g = normal(6, 5, 1, 1, seed=8)
    out = torch.empty(6, 5, 1, 1, device="cuda").as_strided((6, 5, 1, 1), (5, 1, 5, 5))
    assert g.stride() != out.stride()
    norm, (got,) = tg.clip_gradients([g], 1.0, out=[out])
    assert got is out and torch.equal(out, tg.clip_gradients([g], 1.0)[1][0])
    with pytest.raises(ValueError):  # another order
        tg.clip_gradients([normal(6, 5, seed=9)], 1.0, out=[torch.empty(5, 6, device="cuda").t()])


def test_norms_up_to_the_range_of_their_squares():
    """Squares that add up to less than float32's largest value have a finite norm, whichever tensors and blocks they
    lie in; a value whose square is larger has an infinite one, and nothing is clipped."""
    for n, value in ((8192, 1e17), (1 << 22, 8e15), (3, 5e18), (1 << 26, 2e15)):
        grads = [torch.full((n,), value, device="cuda"), torch.full((5,), value, device="cuda")]
        ref = math.sqrt(n + 5) * float(grads[0][0].double())
        assert ref ** 2 < 3.4e38
        norm, out = tg.clip_gradients(grads, ref / 4)
        assert abs(float(norm) - ref) <= 2 ** -20 * ref
        for g, o in zip(grads, out):
            assert ((o - g / 4).abs() <= 2 ** -19 * g / 4).all()
    grads = [torch.tensor([1.0, -1.9e19], device="cuda")]
    norm, out = tg.clip_gradients(grads, 1.0, 2.0)
    assert float(norm) == math.inf and torch.equal(out[0], grads[0] / 2)
