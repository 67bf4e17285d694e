"""Gradients unscaled and clipped by their global norm on the GPU, against 64 bits.

Tolerances.  A square's rounding is 2^-24 of it; a thread adds at most n / 64 squares of each of its four
sums one after the other (a chunk has 32 values a thread), at worst cut 2^-24 a step, and a block's sums meet in
float32: within (n / 64 + 64) 2^-24 of the sum of squares, half of that for the norm, and a rounding.  The
outputs are off by the factor's error, one product and one rounding to their type.
"""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import D64, _built, gen  # noqa: E402,F401


def gradients(shapes, seed, dtypes=(torch.float16, torch.float32), size=1.0):
    g = gen(seed)
    return [(torch.randn(s, generator=g, device="cuda") * size).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(shapes)]


def check(grads, max_norm, scale, norm, out):
    n = sum(g.numel() for g in grads)
    ref = math.sqrt(sum(float(g.to(D64).square().sum()) for g in grads)) / scale
    off = (n / 64 + 64) * 2 ** -25 + 2 ** -23
    assert norm.shape == () and norm.dtype == torch.float32
    assert abs(float(norm) - ref) <= off * ref
    if out is None:
        return
    f = min(1.0, max_norm / ref) / scale if ref > 0 else 1 / scale
    for g, o in zip(grads, out):
        want = g.to(D64) * f
        half = torch.finfo(o.dtype).eps / 2
        tol = (off + half + 2 ** -22) * want.abs() + (2 ** -25 if o.dtype == torch.float16 else 2 ** -149)
        assert o.shape == g.shape and ((o.to(D64) - want).abs() <= tol).all()


SHAPES = [[(1,)], [(7,), (3, 5)], [(8192,), (8193,), (1,)], [(0,), (5, 0), (33,)],
          [(1000, 37), (64,), (64,), (129, 513), (8, 8, 8), (), (2047,)], [(3000, 4099)],
          [(i % 50 + 1, 17) for i in range(700)]]


@pytest.mark.parametrize("dtypes", [(torch.float16,), (torch.float32,), (torch.float16, torch.float32)])
@pytest.mark.parametrize("shapes", SHAPES)
def test_clip(shapes, dtypes):
    grads = gradients(shapes, 1, dtypes)
    size = math.sqrt(sum(float(g.to(D64).square().sum()) for g in grads))
    before = [g.clone() for g in grads]
    for max_norm, scale in ((0.3 * size, 1.0), (0.01 * size / 64, 64.0), (2 * size, 1.0), (math.inf, 8.0), (0.0, 1.0)):
        norm, out = tg.clip_gradients(grads, max_norm, scale)
        assert all(o.dtype == torch.float32 for o in out)
        check(grads, max_norm, scale, norm, out)
    check(grads, 0, 4.0, tg.gradient_norm(grads, 4.0), None)
    assert all(torch.equal(a, b) for a, b in zip(before, grads))
    half = [torch.empty_like(g, dtype=torch.float16) for g in grads]
    norm, out = tg.clip_gradients(grads, 0.5 * size, out=half)
    assert all(a is b for a, b in zip(out, half))
    check(grads, 0.5 * size, 1.0, norm, out)
    norm, out = tg.clip_gradients(grads, 0.5 * size, out=grads)  # in place
    check(before, 0.5 * size, 1.0, norm, out)


@pytest.mark.parametrize("offset", [0, 1, 3, 4, 8])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_alignment(offset, dtype):
    """Views that start anywhere; what lies beside them stays."""
    for n in (1, 5, 20000):
        buf = (torch.randn(n + 40, generator=gen(2), device="cuda")).to(dtype)
        out = torch.full((n + 40,), 9.0, device="cuda")
        for o in (offset, 0):
            dst = out[o:o + n]
            norm, _ = tg.clip_gradients([buf[offset:offset + n]], 0.1, 2.0, out=[dst])
            check([buf[offset:offset + n]], 0.1, 2.0, norm, [dst])
            assert (out[o + n:] == 9).all() and (out[:o] == 9).all()
            out.fill_(9.0)


def test_orders_of_memory():
    g = torch.randn(30, 50, generator=gen(3), device="cuda").half()
    grads = [g.t(), torch.randn(2, 3, 4, 5, generator=gen(4), device="cuda").to(memory_format=torch.channels_last)]
    norm, out = tg.clip_gradients(grads, 1.0)
    check(grads, 1.0, 1.0, norm, out)
    assert all(a.stride() == b.stride() for a, b in zip(out, grads))


def test_not_finite():
    """A norm that is not finite clips nothing: what overflowed stays where it is."""
    for value in (math.inf, -math.inf, math.nan):
        grads = gradients([(100, 33), (7,)], 5)
        grads[0][50, 3] = value
        norm, out = tg.clip_gradients(grads, 0.5, 4.0)
        assert not math.isfinite(float(norm))
        for g, o in zip(grads, out):
            assert torch.equal(torch.nan_to_num(o), torch.nan_to_num(g.float() / 4))
            assert torch.equal(o.isfinite(), g.isfinite())
    norm, out = tg.clip_gradients([torch.zeros(40, device="cuda")], 1.0)
    assert float(norm) == 0 and (out[0] == 0).all()


def test_long_tensor():
    """More than 2^31 elements."""
    n = 2 ** 31 + 12345
    g = torch.empty(n, dtype=torch.float16, device="cuda")
    g.fill_(0.5)
    g[-1] = 300.0
    norm, (out,) = tg.clip_gradients([g], 1.0, 2.0, out=[g])
    ref = math.sqrt((n - 1) * 0.25 + 9e4) / 2
    assert abs(float(norm) - ref) <= 1e-5 * ref
    for i in (0, 2 ** 31 - 1, 2 ** 31, n - 2):
        assert abs(float(g[i]) - 0.25 / ref) <= 2 ** -10 * 0.25 / ref + 2 ** -24
    assert abs(float(g[-1]) - 150 / ref) <= 2 ** -9 * 150 / ref


def test_same_bits_again_captured_and_on_a_stream():
    grads = gradients([(300, 1000), (70,), (4096, 512)], 6)
    want = tg.clip_gradients(grads, 10.0, 16.0)
    again = tg.clip_gradients(grads, 10.0, 16.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tg.clip_gradients(grads, 10.0, 16.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tg.clip_gradients(grads, 10.0, 16.0)
    got[0].zero_()
    for t in got[1]:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for r in (again, other, got):
        assert torch.equal(r[0], want[0]) and all(torch.equal(a, b) for a, b in zip(r[1], want[1]))


def test_refusals():
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda").half()
    for grads, kind in ([], ValueError), ([a.cpu()], ValueError), ([a.double()], TypeError), \
            ([torch.ones(8, 8, device="cuda")[:, :4]], ValueError), ([a[::2]], ValueError), \
            ([a[:1].expand(4)], ValueError):
        with pytest.raises(kind):
            tg.clip_gradients(grads, 1.0)
    for out in ([a], [a, a], [a, b.double()], [a[:32], b], [a, a[:64].view(8, 8)]):
        with pytest.raises((ValueError, TypeError, tg.TgError)):
            tg.clip_gradients([a, b], 1.0, out=out)
    for out in ([a, a], [b, b]):  # written twice
        with pytest.raises(tg.TgError):
            tg.clip_gradients([b, b], 1.0, out=out)
    buf = torch.ones(100, device="cuda")
    with pytest.raises(tg.TgError):  # an output over another gradient
        tg.clip_gradients([buf[:50], buf[50:]], 1.0, out=[buf[40:90], torch.empty(50, device="cuda")])
    with pytest.raises(tg.TgError):  # or over its own, not exactly
        tg.clip_gradients([buf[:50]], 1.0, out=[buf[8:58]])
    with pytest.raises(ValueError):
        tg.clip_gradients([a], 1.0, out=[torch.ones(64, device="cuda", requires_grad=True)])
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(max_norm=1.0, loss_scale=0.0),
               dict(max_norm=1.0, loss_scale=math.inf)):
        with pytest.raises(tg.TgError):
            tg.clip_gradients([a], **kw)
    norm, out = tg.clip_gradients([a, a], 1.0)  # read twice
    assert abs(float(norm) - math.sqrt(128)) < 1e-5 and torch.equal(out[0], out[1])
