"""The gated feed-forward product and its backward pass on the GPU against their formulas in 64 bits.

Tolerances.  A pre-activation is a float32 sum of K exact products: within e = K 2^-23 sum_k |x_k w_k|
whatever the order, even if every partial sum is cut off.  The activations' slopes are at most 1.13 in
size, and their float32 evaluation is within 2^-18 |act(g)| + 2^-21 |g| (an exponential of up to 20 is within
2^-18 of itself, 1 + erf and 1 + tanh within 2^-22), so
    |h - ref| <= 1.13 eg (|u| + eu) + |act(g)| eu + (2^-18 |act(g)| + 2^-21 |g|) (|u| + eu) + rounding,
the rounding to fp16 being 2^-11 of the value (all of the above included) and 2^-25 below its smallest
normal numbers.  Backward, from given gate and up: dG = dh u act'(g) is within 2^-11 of itself and 2^-25
(its rounding to fp16) and 2^-18 |dh u| (the slope), dU likewise with act(g); the products add up those
times the other operand, their own sums (n terms: n 2^-23 of the sum of magnitudes) and a rounding.
"""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402
from tests.test_gpu_head import gen, rows  # noqa: E402

D64 = torch.float64
ACTS = {"none": tg.TG_ACT_NONE, "relu": tg.TG_ACT_RELU, "gelu": tg.TG_ACT_GELU,
        "gelu_tanh": tg.TG_ACT_GELU_TANH, "silu": tg.TG_ACT_SILU}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp16_gemm_relu_gb300 import build

    build.build()
    binding.load_library()
    torch.cuda.set_device(0)
    yield
    st, word = binding.tg_device_error_check(clear=True)
    assert st == binding.TG_OK, f"device error word {word:#x}"


def act64(v, name):
    """The activation and its derivative in 64 bits."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        on = (v > 0).to(v.dtype)
        return v * on, on
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def operands(M, N, K, trans, seed, pad=0, offset=0):
    g = gen(seed)
    x = rows(torch.randn(M, K, generator=g, device="cuda"), pad, offset)
    ws = []
    for _ in range(2):
        w = torch.randn(K, N, generator=g, device="cuda") * (1.5 / math.sqrt(K))
        ws.append(rows(w.t() if trans else w, pad, offset))
    return x, *ws


def rounded(got, ref, err, what=""):
    tol = err + 2 ** -11 * (ref.abs() + err) + 2 ** -25
    assert got.shape == ref.shape and got.dtype == torch.float16
    bad = ~((got.to(D64) - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got.to(D64) - ref).abs() - tol).max()))


def check_forward(x, wg, wu, trans, act, h, gate=None, up=None):
    xd = x.to(D64)
    wgd, wud = ((w.t() if trans else w).to(D64) for w in (wg, wu))
    K = xd.shape[1]
    g, u = xd @ wgd, xd @ wud
    eg, eu = (K * 2 ** -23 * (xd.abs() @ w.abs()) for w in (wgd, wud))
    a = act64(g, act)[0]
    err = (1.13 * eg * (u.abs() + eu) + a.abs() * eu
           + (2 ** -18 * a.abs() + 2 ** -21 * g.abs()) * (u.abs() + eu))
    rounded(h, a * u, err, "h")
    if gate is not None:
        rounded(gate, g, eg, "gate")
        rounded(up, u, eu, "up")


def check_backward(dh, x, wg, wu, gate, up, trans, act, dx, dwg, dwu):
    d, xd, g, u = (t.to(D64) for t in (dh, x, gate, up))
    wgd, wud = ((w.t() if trans else w).to(D64) for w in (wg, wu))
    a, s = act64(g, act)
    dG, dU = d * u * s, d * a
    eG = 2 ** -11 * dG.abs() + 2 ** -25 + 2 ** -18 * (d * u).abs()
    eU = 2 ** -11 * dU.abs() + 2 ** -25 + (2 ** -18 * a.abs() + 2 ** -21 * g.abs()) * d.abs()
    M, N = d.shape
    n = 2 ** -23

    if dx is not None:
        ref = dG @ wgd.t() + dU @ wud.t()
        mag = dG.abs() @ wgd.abs().t() + dU.abs() @ wud.abs().t()
        rounded(dx, ref, eG @ wgd.abs().t() + eU @ wud.abs().t() + (2 * N + 8) * n * mag, "dx")
    for got, full, e in ((dwg, dG, eG), (dwu, dU, eU)):
        if got is not None:
            rounded(got.t() if trans else got, xd.t() @ full,
                    xd.abs().t() @ e + (M + 8) * n * (xd.abs().t() @ full.abs()), "dw")


SIZES = [(1, 1, 1), (1, 8, 8), (2, 7, 3), (1, 640, 512), (3, 257, 200), (17, 100, 65), (64, 1000, 520),
         (65, 129, 1030), (128, 128, 64), (129, 513, 72), (130, 255, 257), (256, 384, 128),
         (300, 2048, 640), (513, 777, 130), (700, 640, 1088)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K, trans):
    x, wg, wu = operands(M, N, K, trans, 1)
    check_forward(x, wg, wu, trans, "silu", tg.gated_linear(x, wg, wu, trans_w=trans))
    h, gate, up = tg.gated_linear(x, wg, wu, tg.TG_ACT_GELU_TANH, trans_w=trans, keep=True)
    check_forward(x, wg, wu, trans, "gelu_tanh", h, gate, up)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K,pad,offset", [
    (5, 72, 40, 3, 1), (140, 200, 136, 8, 0), (140, 200, 136, 8, 8), (90, 333, 77, 1, 5), (300, 300, 300, 4, 2)])
def test_activations_and_strides(M, N, K, pad, offset, trans, act):
    x, wg, wu = operands(M, N, K, trans, 2, pad, offset)
    h, gate, up = tg.gated_linear(x, wg, wu, ACTS[act], trans_w=trans, keep=True)
    check_forward(x, wg, wu, trans, act, h, gate, up)
    dh = rows(torch.randn(M, N, generator=gen(3), device="cuda") * 0.25, pad, offset)
    check_backward(dh, x, wg, wu, gate, up, trans, act,
                   *tg.gated_linear_backward(dh, x, wg, wu, gate, up, ACTS[act], trans_w=trans))


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_backward(M, N, K, trans):
    x, wg, wu = operands(M, N, K, trans, 4)
    _, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
    dh = (torch.randn(M, N, generator=gen(5), device="cuda") * 0.25).half()
    got = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
    check_backward(dh, x, wg, wu, gate, up, trans, "silu", *got)
    dx, none, none_too = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans,
                                                  weight_grads=False)
    assert none is None and none_too is None  # (alone, dX may be summed in other splits)
    check_backward(dh, x, wg, wu, gate, up, trans, "silu", dx, None, None)
    none, dwg, dwu = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, input_grad=False)
    assert none is None and torch.equal(dwg, got[1]) and torch.equal(dwu, got[2])


@pytest.mark.parametrize("trans", [False, True])
def test_weights_in_one_buffer(trans):
    """Both weights as halves of one tensor, and out as a slice of a wider buffer."""
    M, N, K = 200, 320, 256
    both = (torch.randn(K, 2 * N, generator=gen(6), device="cuda") * 0.1).half()
    both = both.t().contiguous() if trans else both
    wg, wu = (both[:N], both[N:]) if trans else (both[:, :N], both[:, N:])
    x = torch.randn(M, K, generator=gen(7), device="cuda").half()
    wide = torch.full((M, N + 24), 7.0, dtype=torch.float16, device="cuda")
    for first in (0, 8, 3):
        out = wide[:, first:first + N]
        assert tg.gated_linear(x, wg, wu, trans_w=trans, out=out) is out
        check_forward(x, wg, wu, trans, "silu", out)
        assert (wide[:, first + N:] == 7).all()
        wide.fill_(7.0)


@pytest.mark.parametrize("options", [
    dict(block_n=128, pair=-1), dict(block_n=256, pair=-1), dict(pair=1), dict(split_k=3, pair=-1),
    dict(split_k=2, pair=1), dict(split_k=5, block_n=256, pair=-1), dict(max_ctas=4), dict(panel_m=2)])
@pytest.mark.parametrize("M,N,K", [(40, 520, 1000), (600, 392, 712), (261, 1027, 330)])
@pytest.mark.parametrize("trans", [False, True])
def test_plans(M, N, K, trans, options):
    x, wg, wu = operands(M, N, K, trans, 8)
    h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True, options=options)
    check_forward(x, wg, wu, trans, "silu", h, gate, up)


def test_empty_batch():
    x = torch.empty(0, 40, dtype=torch.float16, device="cuda")
    w = torch.ones(40, 24, dtype=torch.float16, device="cuda")
    h, gate, up = tg.gated_linear(x, w, w, keep=True)
    assert h.shape == gate.shape == up.shape == (0, 24)
    dx, dwg, dwu = tg.gated_linear_backward(h, x, w, w, gate, up)
    assert dx.shape == (0, 40) and (dwg == 0).all() and (dwu == 0).all() and dwg.shape == w.shape


@pytest.mark.parametrize("act", list(ACTS))
def test_extreme_gates(act):
    """Gates far on either side, at the type's largest values, infinite and NaN: where the value or slope
    has a limit, that is what comes out."""
    g = torch.tensor([-65504.0, -300, -90, -17, -1e-7, 0.0, 1e-7, 17, 90, 300, 65504, -math.inf, math.inf],
                     device="cuda").half()
    n = g.shape[0]
    up, dh = torch.full_like(g, 0.5), torch.ones_like(g)
    eye = torch.eye(n, device="cuda").half()  # dw = x^T dG with x one row of ones
    x = torch.ones(1, n, device="cuda").half()
    dx, dwg, _ = tg.gated_linear_backward(dh[None], x, eye, eye, g[None], up[None], ACTS[act])
    slope = act64(g[:11].to(D64), act)[1] * 0.5
    assert ((dwg[0, :11].to(D64) - slope).abs() <= 2 ** -10 * slope.abs() + 2 ** -18).all()
    limit = 0.5 if act == "none" else 0.0
    assert dwg[0, 11] == limit and dwg[0, 12] == 0.5
    nan = torch.full((1, n), math.nan, device="cuda").half()
    dwg = tg.gated_linear_backward(dh[None], x, eye, eye, nan, up[None], ACTS[act])[1]
    assert (dwg == 0).all() if act == "relu" else (dwg == 0.5).all() if act == "none" else dwg.isnan().all()


def test_rows_do_not_meet():
    """A row of NaN or infinities shows in that row alone."""
    M, N, K = 300, 264, 136
    x, wg, wu = operands(M, N, K, False, 9)
    want = tg.gated_linear(x, wg, wu, keep=True)
    bad = x.clone()
    bad[7], bad[200] = math.nan, math.inf
    got = tg.gated_linear(bad, wg, wu, keep=True)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[7, 200]] = False
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep]) and b[7].isnan().all()


def test_long_hidden_and_offsets():
    """Sums longer than one accumulator takes, and outputs past 2^31 bytes."""
    M, N, K = 33, 40000, 72
    x, wg, wu = operands(M, N, K, True, 10)
    _, gate, up = tg.gated_linear(x, wg, wu, trans_w=True, keep=True)
    dh = (torch.randn(M, N, generator=gen(11), device="cuda") * 0.25).half()
    check_backward(dh, x, wg, wu, gate, up, True, "silu",
                   *tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=True))
    M, N, K = 70000, 16640, 8
    x, wg, wu = operands(M, N, K, False, 12)
    h = tg.gated_linear(x, wg, wu)
    check_forward(x[-300:], wg, wu, False, "silu", h[-300:])
    check_forward(x[:300], wg, wu, False, "silu", h[:300])


def test_same_bits_again_captured_and_on_a_stream():
    M, N, K = 200, 1000, 600
    x, wg, wu = operands(M, N, K, False, 13)
    dh = (torch.randn(M, N, generator=gen(14), device="cuda") * 0.25).half()

    def step():
        h, gate, up = tg.gated_linear(x, wg, wu, keep=True)
        return h, gate, up, *tg.gated_linear_backward(dh, x, wg, wu, gate, up)

    want = step()
    for a, b in zip(want, step()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = tg.gated_linear(x, wg, wu, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(h, want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", list(ACTS))
def test_autograd(act):
    M, N, K = 96, 200, 136
    x, wg, wu = (t.clone().requires_grad_(True) for t in operands(M, N, K, False, 15))
    h = autograd.gated_linear(x, wg, wu, ACTS[act])
    dh = (torch.randn(M, N, generator=gen(16), device="cuda") * 0.25).half()
    h.backward(dh)
    with torch.no_grad():
        _, gate, up = tg.gated_linear(x, wg, wu, ACTS[act], keep=True)
    check_backward(dh, x.detach(), wg.detach(), wu.detach(), gate, up, False, act, x.grad, wg.grad,
                   wu.grad)
    x.grad = None
    h = autograd.gated_linear(x, wg.detach(), wu.detach(), ACTS[act])
    only, = torch.autograd.grad(h, x, dh, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        only.float().sum().backward()


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_autograd_without_gradients(off):
    """Parameters in a serving loop: nothing is kept, and the product is the same."""
    M, N, K = 1024, 4096, 128
    x, wg, wu = operands(M, N, K, False, 19)
    want = tg.gated_linear(x, wg, wu)
    wg, wu = torch.nn.Parameter(wg), torch.nn.Parameter(wu)
    with off():
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        got = autograd.gated_linear(x, wg, wu)
        used = torch.cuda.max_memory_allocated() - before
    assert torch.equal(got, want) and not got.requires_grad and used < 2 * want.nbytes


def test_differences():
    """The gradient against differences of the loss sum(dh h), along directions that keep fp16's grid:
    each step moves the operands by whole multiples of their spacing."""
    M, N, K = 16, 48, 32
    x, wg, wu = operands(M, N, K, False, 17)
    dh = (torch.randn(M, N, generator=gen(18), device="cuda") * 0.25).half()
    _, gate, up = tg.gated_linear(x, wg, wu, keep=True)
    grads = tg.gated_linear_backward(dh, x, wg, wu, gate, up)

    def loss(x, wg, wu):  # of the operator's float32 sums, by the formula in 64 bits
        g, u = x.to(D64) @ wg.to(D64), x.to(D64) @ wu.to(D64)
        return (dh.to(D64) * act64(g, "silu")[0] * u).sum()

    for i, t in enumerate((x, wg, wu)):
        way = torch.randn(t.shape, generator=gen(19 + i), device="cuda").to(D64)
        eps = 1e-5
        moved = [[a.to(D64) + (s * eps * way if j == i else 0) for j, a in enumerate((x, wg, wu))]
                 for s in (1, -1)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / (2 * eps)
        got = (grads[i].to(D64) * way).sum()
        # each gradient is within 2^-9 of its size (kept pre-activations, dG and the result rounded)
        assert (got - slope).abs() <= 2 ** -9 * (grads[i].to(D64) * way).abs().sum()


def test_refusals():
    x, wg, wu = operands(8, 24, 16, False, 20)
    for args, kind in [((x.float(), wg, wu), TypeError), ((x.cpu(), wg, wu), ValueError),
                       ((x, wg[:, :8], wu), ValueError), ((x[:, :8], wg, wu), ValueError),
                       ((x, wg.t(), wu.t()), ValueError), ((x[0], wg, wu), ValueError)]:
        with pytest.raises(kind):
            tg.gated_linear(*args)
    with pytest.raises(tg.TgError):
        tg.gated_linear(x, wg, wu, activation=9)
    with pytest.raises(ValueError):
        tg.gated_linear(x, wg, wu, out=torch.empty(8, 23, dtype=torch.float16, device="cuda"))
    leaf = torch.zeros(8, 24, dtype=torch.float16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        tg.gated_linear(x, wg, wu, out=leaf)
    h, gate, up = tg.gated_linear(x, wg, wu, keep=True)
    with pytest.raises(ValueError):
        tg.gated_linear_backward(h, x, wg, wu, gate[:4], up)
    for options in (dict(block_n=192), dict(block_n=100), dict(split_k=-1), dict(pair=2), dict(force_repack=1),
                    dict(pair=1, max_ctas=1)):
        with pytest.raises(tg.TgError):
            tg.gated_linear(x, wg, wu, options=options)
        for which in (dict(), dict(input_grad=False), dict(weight_grads=False)):
            with pytest.raises(tg.TgError):
                tg.gated_linear_backward(h, x, wg, wu, gate, up, options=options, **which)
