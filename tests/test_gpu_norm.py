"""Layer normalisation on the GPU, forward and backward, against the definition in 64 bits.

Tolerances.  A row's sums run over at most 32 values a thread in order, then 10 halvings: at most 42
float32 roundings, relative error below 2^-18.6 of the sum of magnitudes.  So a mean is within
2^-18 mean|x|, rstd within 2^-17 of itself (eps aside), and y within
    2^-11 |y| + 2^-25                                     its rounding to fp16 (or subnormal spacing)
  + 2^-16 ((|x| + mean|x|) rstd |gamma| + |beta|)         the float32 arithmetic.
dx carries the same per-term errors through g, h mean(g h) and mean(g); dgamma and dbeta are float32
sums of `rows` terms in at most rows / 16 + 64 additions in order (a thread's rows, then partials).
"""

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp16_gemm_relu_gb300 import build

    build.build()
    binding.load_library()
    torch.cuda.set_device(0)
    yield
    st, word = binding.tg_device_error_check(clear=True)
    assert st == binding.TG_OK, f"device error word {word:#x}"


def make(M, N, pad=0, offset=0, seed=0, scale=1.0, shift=0.0):
    """(M, N) fp16 rows of a buffer of N + pad columns, its first element `offset` elements in;
    everything around the rows is NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + M * 31 + N)
    buf = torch.full((offset + M * (N + pad) + 8,), float("nan"), dtype=torch.float16,
                     device="cuda")
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(torch.randn(M, N, generator=g, device="cuda") * scale + shift)
    return view


def reference(x, gamma, beta):
    d = torch.float64
    xd = x.to(d)
    mean = xd.mean(1)
    rstd = 1 / torch.sqrt(((xd - mean[:, None]) ** 2).mean(1) + EPS)
    h = (xd - mean[:, None]) * rstd[:, None]
    y = h * (gamma.to(d) if gamma is not None else 1) + (beta.to(d) if beta is not None else 0)
    return y, mean, rstd, h


def check_forward(x, gamma, beta, y, mean, rstd):
    yr, mr, rr, _ = reference(x, gamma, beta)
    xd = x.double().abs()
    size = xd.mean(1)
    ga = gamma.double().abs() if gamma is not None else 1.0
    ba = beta.double().abs() if beta is not None else 0.0
    tol = yr.abs() * 2 ** -11 + 2 ** -25 + 2 ** -16 * ((xd + size[:, None]) * rr[:, None] * ga + ba)
    assert ((y.double() - yr).abs() <= tol).all()
    assert ((mean.double() - mr).abs() <= 2 ** -18 * size + 1e-30).all()
    # the mean's error enters the variance squared, beside the sum's own
    assert ((rstd.double() - rr).abs() <= rr * (2 ** -17 + (2 ** -18 * size * rr) ** 2)).all()


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 8), (2, 31), (9, 64), (300, 65), (33, 256), (4, 257),
          (17, 1000), (8, 1024), (5, 2047), (3, 2048), (2, 4096), (7, 3073), (2, 8192), (3, 12345),
          (1, 16384), (2, 16385), (1, 32768), (2, 32767)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (5, 0), (0, 3), (8, 1), (1, 7)])
def test_forward(M, N, pad, offset):
    x = make(M, N, pad, offset, 1, 2.0, 0.5)
    gamma, beta = make(1, N, seed=2)[0].contiguous(), make(1, N, seed=3)[0].contiguous()
    buf = torch.full((M, N + 9), 7.0, dtype=torch.float16, device="cuda")
    out = buf[:, offset:offset + N]  # other alignments than x's, and columns to leave alone
    y, mean, rstd = tg.layer_norm(x, gamma, beta, eps=EPS, stats=True, out=out)
    assert y is out
    check_forward(x, gamma, beta, y, mean, rstd)
    assert (buf[:, :offset] == 7).all() and (buf[:, offset + N:] == 7).all()
    # an output at another alignment may go by another order of the sums
    check_forward(x, gamma, beta, tg.layer_norm(x, gamma, beta, eps=EPS), mean, rstd)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("which", ["both", "gamma", "beta", "none"])
def test_forward_parameters(dtype, which):
    x = make(37, 520, 3, 0, 4)
    gamma = make(1, 520, seed=5)[0].to(dtype).contiguous() if which in ("both", "gamma") else None
    beta = make(1, 520, seed=6)[0].to(dtype).contiguous() if which in ("both", "beta") else None
    y, mean, rstd = tg.layer_norm(x, gamma, beta, eps=EPS, stats=True)
    check_forward(x, gamma, beta, y, mean, rstd)


def test_parameters_at_any_alignment():
    gamma = make(1, 1001, offset=1, seed=7)[0]
    beta = make(1, 1001, offset=3, seed=8)[0]
    x, dy = make(9, 1001, seed=9), make(9, 1001, seed=10)
    y, mean, rstd = tg.layer_norm(x, gamma, beta, eps=EPS, stats=True)
    check_forward(x, gamma, beta, y, mean, rstd)
    check_backward(dy, x, gamma, mean, rstd, *tg.layer_norm_backward(dy, x, mean, rstd, gamma))


def test_forward_large_offset_and_extremes():
    # a mean far larger than the spread: the variance must not cancel
    x = make(5, 4096, seed=11, scale=0.5, shift=1000.0)
    y, mean, rstd = tg.layer_norm(x, eps=EPS, stats=True)
    check_forward(x, None, None, y, mean, rstd)
    # a constant row has variance 0; rows of the largest fp16 values do not overflow float32
    x = torch.full((2, 777), 3.0, dtype=torch.float16, device="cuda")
    x[1, ::2], x[1, 1::2] = 65504.0, -65504.0
    y, mean, rstd = tg.layer_norm(x, eps=EPS, stats=True)
    check_forward(x, None, None, y, mean, rstd)
    assert (y[0] == 0).all()
    # a NaN or an infinity stays in its own row
    x = make(4, 100, seed=12).clone()
    x[1, 5], x[2, 6] = float("nan"), float("inf")
    y = tg.layer_norm(x, eps=EPS)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()


def test_forward_in_place():
    for pad in (0, 3):
        x = make(50, 1003, pad, seed=13)
        want = tg.layer_norm(x, eps=EPS, out=torch.empty_strided(
            x.shape, x.stride(), dtype=x.dtype, device="cuda"))
        got = tg.layer_norm(x, eps=EPS, out=x)
        assert got is x and torch.equal(x, want)


def backward_reference(dy, x, gamma, mean, rstd):
    d = torch.float64
    h = (x.to(d) - mean.to(d)[:, None]) * rstd.to(d)[:, None]
    dyd = dy.to(d)
    g = dyd * (gamma.to(d) if gamma is not None else 1)
    b = (g * h).mean(1, keepdim=True)
    dx = rstd.to(d)[:, None] * (g - g.mean(1, keepdim=True) - h * b)
    return dx, (dyd * h).sum(0), dyd.sum(0), h, g


def check_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta):
    M = x.shape[0]
    dxr, dgr, dbr, h, g = backward_reference(dy, x, gamma, mean, rstd)
    # h as computed: (x - mean) rounded, times rstd
    he = h.abs() * 2 ** -22
    terms = g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True)
    extra = rstd.double()[:, None] * 2 ** -16 * terms
    assert ((dx.double() - dxr).abs() <= dxr.abs() * 2 ** -11 + 2 ** -25 + extra).all()
    adds = (M / 16 + 64) * 2 ** -24
    last = 2 ** -11 if (gamma is not None and gamma.dtype == torch.float16) else 2 ** -24
    small = 2 ** -25 if last == 2 ** -11 else 1e-37
    dya = dy.double().abs()
    tol_g = dgr.abs() * last + small + (dya * (h.abs() * (adds + 2 ** -22) + he)).sum(0)
    tol_b = dbr.abs() * last + small + dya.sum(0) * adds
    assert ((dgamma.double() - dgr).abs() <= tol_g).all()
    assert ((dbeta.double() - dbr).abs() <= tol_b).all()


@pytest.mark.parametrize("M,N", SHAPES + [(1000, 64), (5000, 40), (700, 3073), (2000, 520)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (5, 0), (8, 1)])
def test_backward(M, N, pad, offset):
    x, dy = make(M, N, pad, offset, 20, 1.5, 0.3), make(M, N, pad + 2, offset, 21)
    gamma = make(1, N, seed=22)[0].contiguous()
    _, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
    got = tg.layer_norm_backward(dy, x, mean, rstd, gamma)
    assert got[1].dtype == got[2].dtype == torch.float16
    check_backward(dy, x, gamma, mean, rstd, *got)
    again = tg.layer_norm_backward(dy, x, mean, rstd, gamma)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.float32, None])
def test_backward_parameter_types(dtype):
    x, dy = make(333, 777, seed=23), make(333, 777, seed=24)
    gamma = make(1, 777, seed=25)[0].to(dtype).contiguous() if dtype else None
    _, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
    got = tg.layer_norm_backward(dy, x, mean, rstd, gamma)
    assert got[1].dtype == torch.float32
    check_backward(dy, x, gamma, mean, rstd, *got)
    dx, none1, none2 = tg.layer_norm_backward(dy, x, mean, rstd, gamma, param_grads=False)
    assert none1 is None and none2 is None and torch.equal(dx, got[0])


@pytest.mark.parametrize("M,N", [(700, 60), (40, 500), (300, 1000), (50, 4097), (9, 9000), (5, 20000)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
@pytest.mark.parametrize("over", ["dy", "x"])
def test_backward_in_place(M, N, pad, offset, over):
    # the C entry may write dX over dY or X; N in every range of the kernels
    x, dy = make(M, N, pad, offset, 32, 1.5, 0.3), make(M, N, pad, offset, 33)
    gamma = make(1, N, seed=34)[0].contiguous()
    _, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
    keep_x, keep_dy = x.clone(), dy.clone()
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    out = dy if over == "dy" else x
    st = binding.tg_layernorm_backward_f16(
        dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        out.data_ptr(), dg.data_ptr(), db.data_ptr(), M, N, dy.stride(0), x.stride(0),
        out.stride(0), binding.TG_TYPE_F16, torch.cuda.current_stream().cuda_stream)
    assert st == binding.TG_OK
    check_backward(keep_dy, keep_x, gamma, mean, rstd, out, dg, db)
    # each output alone, and none of the others touched
    alone = torch.empty_like(gamma)
    st = binding.tg_layernorm_backward_f16(
        keep_dy.data_ptr(), keep_x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        0, 0, alone.data_ptr(), M, N, keep_dy.stride(0), keep_x.stride(0), 0, binding.TG_TYPE_F16,
        torch.cuda.current_stream().cuda_stream)
    assert st == binding.TG_OK
    _, _, dbr, _, _ = backward_reference(keep_dy, keep_x, gamma, mean, rstd)
    tol = dbr.abs() * 2 ** -11 + 2 ** -25 + keep_dy.double().abs().sum(0) * (M / 16 + 64) * 2 ** -24
    assert ((alone.double() - dbr).abs() <= tol).all()


@pytest.mark.parametrize("M,N", [(1, 600), (7, 513), (61, 1017), (61, 1018), (30, 2041), (30, 2042),
                                 (700, 1537), (1300, 3073), (40, 4090), (17, 8185), (17, 8186),
                                 (9, 12001), (9, 16377), (9, 16378), (11, 5000), (8, 5001),
                                 (9, 5001), (1201, 5001), (2450, 4097)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (1, 3), (5, 6), (8, 7), (3, 0)])
def test_matrices_that_lie_alike(M, N, pad, offset):
    """Rows that miss a 16-byte boundary, all matrices by the same bytes: NaN around x and dy must
    not enter, and what is around y and dx must stay."""
    def room():
        buf = torch.full((offset + M * (N + pad) + 8,), 7.0, dtype=torch.float16, device="cuda")
        return buf, buf[offset:offset + M * (N + pad)].view(M, N + pad)

    x, dy = make(M, N, pad, offset, 40, 1.5, 0.3), make(M, N, pad, offset, 41)
    gamma, beta = make(1, N, seed=42)[0].contiguous(), make(1, N, seed=43)[0].contiguous()
    buf, y = room()
    _, mean, rstd = tg.layer_norm(x, gamma, beta, eps=EPS, stats=True, out=y[:, :N])
    check_forward(x, gamma, beta, y[:, :N], mean, rstd)
    y[:, :N] = 7.0
    assert (buf == 7).all()
    buf, dx = room()
    dgamma, dbeta = torch.empty(2, N, dtype=torch.float16, device="cuda")
    st = binding.tg_layernorm_backward_f16(
        dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), M, N, N + pad, N + pad, N + pad,
        binding.TG_TYPE_F16, torch.cuda.current_stream().cuda_stream)
    assert st == binding.TG_OK
    check_backward(dy, x, gamma, mean, rstd, dx[:, :N], dgamma, dbeta)
    dx[:, :N] = 7.0
    assert (buf == 7).all()


def test_calls_back_to_back():
    """Calls that share scratch and follow one another without a wait give what they give alone."""
    cases = []
    for k, (M, N, pad) in enumerate([(300, 4096, 0), (5, 700, 3), (1000, 512, 0), (64, 5001, 0),
                                     (2, 20000, 0), (700, 3073, 0), (1, 8192, 0)]):
        x, dy = make(M, N, pad, 0, 50 + k), make(M, N, pad, 0, 60 + k)
        gamma = make(1, N, seed=70 + k)[0].contiguous()
        _, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
        torch.cuda.synchronize()
        want = tg.layer_norm_backward(dy, x, mean, rstd, gamma)
        torch.cuda.synchronize()
        cases.append((dy, x, mean, rstd, gamma, want))
    got = [[tg.layer_norm_backward(*c[:5]) for c in cases] for _ in range(20)]
    torch.cuda.synchronize()
    for run in got:
        for g, c in zip(run, cases):
            assert all(torch.equal(a, b) for a, b in zip(g, c[5]))


def test_many_short_rows():
    # more rows than one wave of warps, widths at the edges of the kernels' ranges
    for N in (1, 8, 256, 257, 512, 513):
        x, dy = make(6000, N, 0, 0, 35), make(6000, N, 0, 0, 36)
        gamma = make(1, N, seed=37)[0].contiguous()
        y, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
        check_forward(x, gamma, None, y, mean, rstd)
        check_backward(dy, x, gamma, mean, rstd, *tg.layer_norm_backward(dy, x, mean, rstd, gamma))


def test_backward_against_differences():
    d = torch.float64
    x, dy = make(6, 200, seed=26), make(6, 200, seed=27)
    gamma, beta = make(1, 200, seed=28)[0].contiguous(), make(1, 200, seed=29)[0].contiguous()
    _, mean, rstd = tg.layer_norm(x, gamma, beta, eps=EPS, stats=True)
    grads = tg.layer_norm_backward(dy, x, mean, rstd, gamma)

    def total(xd, gd, bd):
        mu = xd.mean(1, keepdim=True)
        rs = 1 / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + EPS)
        return (dy.to(d) * ((xd - mu) * rs * gd + bd)).sum()

    args = [x.to(d), gamma.to(d), beta.to(d)]
    for k, grad in enumerate(grads):
        way = torch.randn_like(args[k])
        step = 1e-5
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + step * way, args[k] - step * way
        diff = (total(*up) - total(*down)) / (2 * step)
        got = (grad.to(d) * way).sum()
        # each gradient is within 2^-10 of itself (fp16, and float32 arithmetic well inside that)
        assert (got - diff).abs() <= 2 ** -10 * (grad.to(d).abs() * way.abs()).sum() + 1e-6


def test_empty():
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    assert tg.layer_norm(x).shape == (0, 64)
    s = torch.empty(0, device="cuda")
    dx, dg, db = tg.layer_norm_backward(x, x, s, s, torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()


def test_refusals():
    x = make(4, 64)
    s = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        tg.layer_norm(x.float())
    with pytest.raises(TypeError):
        tg.layer_norm(x, torch.ones(64, device="cuda", dtype=torch.float64))
    with pytest.raises(TypeError):
        tg.layer_norm(x, torch.ones(64, device="cuda"), torch.ones(64, device="cuda").half())
    with pytest.raises(ValueError):
        tg.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        tg.layer_norm(x.t())
    with pytest.raises(ValueError):
        tg.layer_norm(x[0])
    with pytest.raises(ValueError):
        tg.layer_norm(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        tg.layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        tg.layer_norm(x, out=torch.empty((4, 63), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x[:3], x, s, s)
    with pytest.raises(ValueError):
        tg.layer_norm_backward(x, x, s[:3], s)
    with pytest.raises(tg.TgError):
        tg.layer_norm(x, eps=-1.0)
    with pytest.raises(tg.TgError):
        tg.layer_norm(torch.zeros((1, 32769), dtype=torch.float16, device="cuda"))


def test_other_stream():
    side = torch.cuda.Stream()
    x, gamma = make(512, 2048, seed=30), make(1, 2048, seed=31)[0].contiguous()
    want = tg.layer_norm(x, gamma, eps=EPS)
    side.wait_stream(torch.cuda.current_stream())
    got = tg.layer_norm(x, gamma, eps=EPS, stream=side)
    raw = tg.layer_norm(x, gamma, eps=EPS, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)
