"""The head's losses on the GPU (cross entropy and distillation, with their gradients) against the
definitions in 64 bits.

Tolerances.  A logit is a float32 sum of D exact products; whatever the order, and even if every
partial sum is cut off instead of rounded, it is within D 2^-23 sum_k |x_k w_k|: dz below, with the
logit scale.  Then
    |lse - ref|  <= dz + 2^-20 (|ref| + 1)                (a few float32 roundings of lse and exp2)
    |loss - ref| <= 2 dz + 2^-20 (|lse| + |z| + 1)        (weighted by q, and the entropy's terms)
An element of G = w (p - q) is within |w| (p (2 dz + 2^-18) + 2^-11 |p - q|) + max|w| 2^-39: the
exponential's relative error, the rounding to fp16, and below that fp16's subnormal spacing.  dX and
dW add up G's errors times the other operand, their own float32 sums (n terms: n 2^-23 of the sum of
magnitudes), and the rounding to fp16.
"""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402

IGNORE = -100
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(values, pad=0, offset=0):
    """The values as fp16 rows of a wider buffer of NaN, `offset` elements in."""
    M, N = values.shape
    buf = torch.full((offset + M * (N + pad) + 8,), float("nan"), dtype=torch.float16,
                     device="cuda")
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(values)
    return view


def operands(T, V, D, layout, seed, spread=2.0, pad=0, offset=0):
    g = gen(seed)
    x = rows(torch.randn(T, D, generator=g, device="cuda"), pad, offset)
    w = torch.randn(V, D, generator=g, device="cuda") * (spread / math.sqrt(D))
    w = rows(w if layout == tg.TG_HEAD_VOCAB_MAJOR else w.t(), pad, offset)
    return x, w


def check(x, w, layout, scale, q, live, entropy, dloss, loss, lse, dx, dw):
    """q: (T, V) the rows' target distributions in 64 bits; live: rows that count; entropy: sum q log
    q of each row."""
    wv = (w if layout == tg.TG_HEAD_VOCAB_MAJOR else w.t()).to(D64)
    xd = x.to(D64)
    T, D = xd.shape
    V = wv.shape[0]
    z = scale * xd @ wv.t()
    dz = scale * D * 2 ** -23 * (xd.abs() @ wv.abs().t())
    lse_r = torch.logsumexp(z, 1)
    dzm = dz.max(1).values
    if lse is not None:
        assert ((lse.to(D64) - lse_r).abs() <= dzm + 2 ** -20 * (lse_r.abs() + 1)).all()
    zq = (q * z).sum(1)
    loss_r = torch.where(live, entropy + lse_r - zq, torch.zeros_like(lse_r))
    size = lse_r.abs() + (q * z.abs()).sum(1) + entropy.abs() + 1
    assert ((loss.to(D64) - loss_r).abs() <= 2 * dzm + 2 ** -19 * size).all()
    assert (loss[~live] == 0).all()
    if dx is None:
        return
    p = torch.exp(z - lse_r[:, None])
    wt = torch.where(live, dloss.to(D64), torch.zeros_like(lse_r))[:, None]
    G = wt * (p - q)
    dG = (wt.abs() * (p * (2 * dz + 2 ** -18) + 2 ** -18 * q + 2 ** -11 * (p - q).abs())
          + wt.abs().max() * 2 ** -39)
    dG = scale * torch.where(live[:, None], dG, torch.zeros_like(dG))
    G = scale * G
    for got, ref, err, n, mag in (
            (dx, G @ wv, dG @ wv.abs(), V, G.abs() @ wv.abs()),
            (dw if layout == tg.TG_HEAD_VOCAB_MAJOR else dw.t(), G.t() @ xd, dG.t() @ xd.abs(), T,
             G.abs().t() @ xd.abs())):
        tol = err + (n + 8) * 2 ** -23 * mag + 2 ** -11 * ref.abs() + 2 ** -24
        assert got.shape == ref.shape and got.dtype == torch.float16
        bad = ~((got.to(D64) - ref).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), float(((got.to(D64) - ref).abs() - tol).max()))


def targets(T, V, seed, ignored=0.2):
    g = gen(seed)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[torch.rand(T, generator=g, device="cuda") < ignored] = IGNORE
    return t


def one_hot(target, V):
    live = target != IGNORE
    q = torch.zeros(target.shape[0], V, dtype=D64, device="cuda")
    q.scatter_(1, target.clamp_min(0)[:, None], live[:, None].to(D64))
    return q, live


def teacher(T, V, top, seed, dtype):
    g = gen(seed)
    index = torch.rand(T, max(V, top), generator=g, device="cuda").topk(top, dim=1).indices % V
    logits = (torch.randn(T, top, generator=g, device="cuda") * 3 + 10).to(dtype)
    short = torch.rand(T, generator=g, device="cuda")
    length = torch.where(short < 0.3, (short / 0.3 * (top + 1)).long(), top)
    index[torch.arange(top, device="cuda")[None, :] >= length[:, None]] = -1
    return index, logits


def teacher_q(index, logits, tau, V):
    there = (index >= 0) & (logits > -math.inf)
    live = there.any(1)
    u = (logits.to(D64) / tau).masked_fill(~there, -1e300)
    qe = torch.softmax(u, 1) * there
    q = torch.zeros(index.shape[0], V, dtype=D64, device="cuda")
    q.scatter_add_(1, index.clamp_min(0), qe)
    return q, live, -torch.special.entr(qe).sum(1)


SIZES = [(1, 1, 1), (1, 2, 8), (2, 7, 3), (1, 1000, 64), (7, 100, 17), (3, 257, 200),
         (64, 4099, 96), (128, 1000, 520), (129, 513, 8), (130, 255, 257), (300, 2048, 64),
         (513, 777, 130)]


@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_cross_entropy(T, V, D, layout, pad, offset):
    x, w = operands(T, V, D, layout, T + V + D, pad=pad, offset=offset)
    target = targets(T, V, V + 5, 0.2 if T > 2 else 0.0)
    dloss = torch.randn(T, generator=gen(3), device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, target, layout=layout, return_lse=True)
    check(x, w, layout, 1.0, q, live, zero, None, loss, lse, None, None)
    step = tg.linear_cross_entropy_step(x, w, target, dloss, layout=layout)
    check(x, w, layout, 1.0, q, live, zero, dloss, step[0], None, step[1], step[2])
    again = tg.linear_cross_entropy_step(x, w, target, dloss, layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(step, again))


@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("tau,dtype", [(1.0, torch.float16), (2.5, torch.float32)])
def test_distillation(T, V, D, layout, tau, dtype):
    top = min(V, 1 + (T * 7) % 70)
    x, w = operands(T, V, D, layout, T + V + D)
    index, logits = teacher(T, V, top, V + 6, dtype)
    dloss = torch.rand(T, generator=gen(4), device="cuda") + 0.5
    q, live, entropy = teacher_q(index, logits, tau, V)
    loss, lse = tg.linear_distillation(x, w, index, logits, temperature=tau, layout=layout,
                                       return_lse=True)
    check(x, w, layout, 1 / tau, q, live, entropy, None, loss, lse, None, None)
    step = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=tau, layout=layout)
    check(x, w, layout, 1 / tau, q, live, entropy, dloss, step[0], None, step[1], step[2])
    again = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=tau, layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(step, again))


@pytest.mark.parametrize("layout", [tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR])
@pytest.mark.parametrize("piece", [1, 100, 256, 299])
@pytest.mark.parametrize("D", [64, 77])
def test_pieces(layout, piece, D):
    T, V = 300, 1003
    x, w = operands(T, V, D, layout, 50)
    target = targets(T, V, 51)
    dloss = torch.randn(T, generator=gen(52), device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    step = tg.linear_cross_entropy_step(x, w, target, dloss, layout=layout, piece_rows=piece)
    check(x, w, layout, 1.0, q, live, zero, dloss, step[0], None, step[1], step[2])
    index, logits = teacher(T, V, 9, 53, torch.float16)
    q, live, entropy = teacher_q(index, logits, 2.0, V)
    step = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=2.0, layout=layout,
                                       piece_rows=piece)
    check(x, w, layout, 0.5, q, live, entropy, dloss, step[0], None, step[1], step[2])
    again = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=2.0, layout=layout,
                                        piece_rows=piece)
    assert all(torch.equal(a, b) for a, b in zip(step, again))


def test_larger_case():
    T, V, D = 1025, 8200, 512
    x, w = operands(T, V, D, 0, 60)
    target = targets(T, V, 61, 0.05)
    dloss = torch.full((T,), 8.0, device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    step = tg.linear_cross_entropy_step(x, w, target, dloss)
    check(x, w, 0, 1.0, q, live, zero, dloss, step[0], None, step[1], step[2])


@pytest.mark.parametrize("spread,scale", [(60.0, 1.0), (2.0, 30.0), (0.0, 1.0), (2.0, 1e-3)])
def test_sharp_and_flat_logits(spread, scale):
    # logits of hundreds: probabilities of exactly 0 and 1; and all equal
    T, V, D = 70, 900, 128
    x, w = operands(T, V, D, 0, 70, spread)
    target = targets(T, V, 71)
    dloss = torch.rand(T, generator=gen(72), device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, target, logit_scale=scale, return_lse=True)
    check(x, w, 0, scale, q, live, zero, None, loss, lse, None, None)
    step = tg.linear_cross_entropy_step(x, w, target, dloss, logit_scale=scale)
    check(x, w, 0, scale, q, live, zero, dloss, step[0], None, step[1], step[2])


@pytest.mark.parametrize("weights", ["mixed", "tiny", "huge", "zero"])
def test_row_weights(weights):
    T, V, D = 90, 600, 64
    x, w = operands(T, V, D, 0, 80)
    target = targets(T, V, 81)
    g = gen(82)
    dloss = torch.randn(T, generator=g, device="cuda")
    if weights == "mixed":  # over eight orders of magnitude, some zero
        dloss *= 10.0 ** (torch.rand(T, generator=g, device="cuda") * 8 - 6)
        dloss[::7] = 0.0
    elif weights == "tiny":
        dloss *= 1e-30  # every gradient rounds to 0 in fp16
    elif weights == "huge":
        dloss *= 100.0
        dloss[target == IGNORE] = 1e30  # of rows that do not count
    else:
        dloss.zero_()
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    step = tg.linear_cross_entropy_step(x, w, target, dloss)
    check(x, w, 0, 1.0, q, live, zero, dloss, step[0], None, step[1], step[2])
    if weights in ("tiny", "zero"):
        assert (step[1] == 0).all() and (step[2] == 0).all()


def test_rows_that_do_not_count():
    T, V, D = 66, 300, 40
    x, w = operands(T, V, D, 0, 90)
    dloss = torch.full((T,), float("nan"), device="cuda")  # nobody reads it
    target = torch.full((T,), IGNORE, dtype=torch.int64, device="cuda")
    loss, dx, dw = tg.linear_cross_entropy_step(x, w, target, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    index = torch.full((T, 5), -1, dtype=torch.int64, device="cuda")
    logits = torch.full((T, 5), float("nan"), device="cuda")
    loss, dx, dw = tg.linear_distillation_step(x, w, index, logits, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    # entries at -inf have no weight; a row of nothing else has no teacher
    index = torch.arange(5, device="cuda").repeat(T, 1).contiguous()
    logits = torch.full((T, 5), -math.inf, device="cuda")
    logits[: T // 2, 3] = 1.0
    dloss = torch.ones(T, device="cuda")
    q, live, entropy = teacher_q(index, logits, 1.0, V)
    assert int(live.sum()) == T // 2
    loss, dx, dw = tg.linear_distillation_step(x, w, index, logits, dloss)
    check(x, w, 0, 1.0, q, live, entropy, dloss, loss, None, dx, dw)
    # another number can be the one to ignore, inside the vocabulary too
    target = torch.randint(0, V, (T,), generator=gen(91), device="cuda")
    target[::3] = 0
    loss, lse = tg.linear_cross_entropy(x, w, target, ignore_index=0, return_lse=True)
    assert (loss[target == 0] == 0).all() and (loss[target != 0] > 0).all()
    assert torch.isfinite(lse).all()


def test_wrong_targets_are_nan():
    T, V, D = 40, 300, 32
    x, w = operands(T, V, D, 0, 95)
    target = targets(T, V, 96, 0.0)
    good = tg.linear_cross_entropy(x, w, target)
    for wrong in (V, V + 1, -1, -2 ** 62, 2 ** 62):
        t = target.clone()
        t[7] = wrong
        loss, dx, dw = tg.linear_cross_entropy_step(x, w, t, torch.ones(T, device="cuda"))
        rest = torch.arange(T, device="cuda") != 7
        assert torch.isnan(loss[7]) and torch.equal(loss[rest], good[rest])
        assert torch.isnan(dx[7]).all() and torch.isfinite(dx[rest]).all()
        assert torch.isnan(dw).any()
    index, logits = teacher(T, V, 6, 97, torch.float32)
    good = tg.linear_distillation_step(x, w, index, logits, torch.ones(T, device="cuda"))[0]
    for wrong in ("index", "nan", "inf"):
        i, u = index.clone(), logits.clone()
        i[7] = torch.arange(6, device="cuda")
        if wrong == "index":
            i[7, 2] = V
        else:
            u[7, 2] = float(wrong)
        loss, dx, _ = tg.linear_distillation_step(x, w, i, u, torch.ones(T, device="cuda"))
        assert torch.isnan(loss[7]) and torch.equal(loss[rest], good[rest])
        assert torch.isnan(dx[7]).all() and torch.isfinite(dx[rest]).all()


def test_not_finite_rows_stay_in_their_rows():
    T, V, D = 40, 300, 32
    x, w = operands(T, V, D, 0, 98)
    target = targets(T, V, 99, 0.0)
    good = tg.linear_cross_entropy(x, w, target)
    x = x.clone()
    x[3, 4] = float("nan")
    x[5] = float("nan")
    target[5] = IGNORE
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    rest = (torch.arange(T, device="cuda") != 3) & (torch.arange(T, device="cuda") != 5)
    assert torch.isnan(loss[3]) and torch.isnan(lse[3]) and torch.isnan(lse[5]) and loss[5] == 0
    assert torch.equal(loss[rest], good[rest])
    _, dx, _ = tg.linear_cross_entropy_step(x, w, target, torch.ones(T, device="cuda"))
    assert torch.isnan(dx[3]).all() and (dx[5] == 0).all() and torch.isfinite(dx[rest]).all()


def test_infinite_logits():
    # fp16 values whose products leave float32's range do not exist; infinities come with the operands
    T, V, D = 20, 300, 64
    x, w = operands(T, V, D, 0, 126)
    w = w.clone()
    x = x.abs().contiguous()
    target = torch.full((T,), 5, dtype=torch.int64, device="cuda")
    good = tg.linear_cross_entropy(x, w, target)
    w[250] = -math.inf  # a token that cannot be: its logit is -inf, its probability 0
    wz = w.clone()
    wz[250] = 0
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    z = (x.double() @ wz.double().t())
    z[:, 250] = -math.inf
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() <= 1e-5 * (want.abs() + 1)).all()
    assert ((loss.double() - (want - z[:, 5])).abs() <= 1e-5 * (want.abs() + 1)).all()
    assert not torch.equal(loss, good) and torch.isfinite(loss).all()
    target[3] = 250
    assert torch.isposinf(tg.linear_cross_entropy(x, w, target)[3])
    w[250] = math.inf
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    assert torch.isnan(lse).all() and torch.isnan(loss).all()
    w[:] = -math.inf  # no token can be
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    assert torch.isneginf(lse).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("V", [1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 383, 385, 511,
                               513])
@pytest.mark.parametrize("T", [1, 7, 8, 127, 129])
def test_tile_edges(T, V):
    D = 72
    x, w = operands(T, V, D, 0, 127 + V)
    target = targets(T, V, 128, 0.0)
    target[-1] = V - 1  # the last column
    dloss = torch.ones(T, device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    check(x, w, 0, 1.0, q, live, zero, None, loss, lse, None, None)
    step = tg.linear_cross_entropy_step(x, w, target, dloss)
    check(x, w, 0, 1.0, q, live, zero, dloss, step[0], None, step[1], step[2])


@pytest.mark.parametrize("D", [1, 63, 64, 65, 1023, 1024, 1025, 1088, 2048, 2112, 3000])
@pytest.mark.parametrize("T,V", [(5, 300), (300, 600)])
def test_widths_around_the_segments(T, V, D):
    x, w = operands(T, V, D, 0, 129 + D)
    target = targets(T, V, 130)
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    loss, lse = tg.linear_cross_entropy(x, w, target, return_lse=True)
    check(x, w, 0, 1.0, q, live, zero, None, loss, lse, None, None)
    step = tg.linear_cross_entropy_step(x, w, target, torch.ones(T, device="cuda"))
    check(x, w, 0, 1.0, q, live, zero, torch.ones(T, device="cuda"), step[0], None, step[1], step[2])


def test_same_token_twice():
    T, V, D = 33, 200, 48
    x, w = operands(T, V, D, 0, 100)
    index = torch.randint(0, 5, (T, 12), generator=gen(101), device="cuda")
    logits = torch.randn(T, 12, generator=gen(102), device="cuda")
    dloss = torch.ones(T, device="cuda")
    q, live, entropy = teacher_q(index, logits, 1.0, V)
    step = tg.linear_distillation_step(x, w, index, logits, dloss)
    check(x, w, 0, 1.0, q, live, entropy, dloss, step[0], None, step[1], step[2])


def test_most_entries():
    T, V, D, top = 5, 3000, 64, 1024
    x, w = operands(T, V, D, 0, 103)
    index, logits = teacher(T, V, top, 104, torch.float16)
    dloss = torch.ones(T, device="cuda")
    q, live, entropy = teacher_q(index, logits, 4.0, V)
    step = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=4.0)
    check(x, w, 0, 0.25, q, live, entropy, dloss, step[0], None, step[1], step[2])


def test_no_rows():
    x = torch.empty((0, 24), dtype=torch.float16, device="cuda")
    w = torch.ones((50, 24), dtype=torch.float16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    dloss = torch.empty(0, device="cuda")
    assert tg.linear_cross_entropy(x, w, none).shape == (0,)
    loss, dx, dw = tg.linear_cross_entropy_step(x, w, none, dloss)
    assert loss.shape == (0,) and dx.shape == (0, 24) and (dw == 0).all()
    loss, dx, dw = tg.linear_distillation_step(x, w, none.view(0, 1), dloss.view(0, 1), dloss)
    assert loss.shape == (0,) and dx.shape == (0, 24) and (dw == 0).all()


def test_one_gradient_alone():
    T, V, D = 60, 400, 56
    x, w = operands(T, V, D, 0, 105)
    target = targets(T, V, 106)
    dloss = torch.randn(T, generator=gen(107), device="cuda")
    loss, dx, dw = tg.linear_cross_entropy_step(x, w, target, dloss)
    for want_dx in (True, False):
        got_x, got_w = torch.zeros_like(x).contiguous(), torch.zeros_like(w).contiguous()
        l2 = torch.empty(T, device="cuda")
        st = binding.tg_linear_cross_entropy_f16(
            x.data_ptr(), w.data_ptr(), target.data_ptr(), IGNORE, 1.0, dloss.data_ptr(),
            l2.data_ptr(), 0, got_x.data_ptr() if want_dx else 0,
            0 if want_dx else got_w.data_ptr(), T, V, D, D, D, D, D, None,
            torch.cuda.current_stream().cuda_stream)
        assert st == binding.TG_OK
        assert torch.equal(l2, loss)
        assert torch.equal(got_x, dx) if want_dx else torch.equal(got_w, dw)


def test_gradients_into_rows_of_a_buffer():
    T, V, D = 70, 300, 51
    x, w = operands(T, V, D, 0, 108)
    target = targets(T, V, 109)
    dloss = torch.randn(T, generator=gen(110), device="cuda")
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    loss = torch.empty(T, device="cuda")
    for pad, offset in ((13, 0), (0, 1), (5, 8)):
        bx = torch.full((T, D + pad + offset), 7.0, dtype=torch.float16, device="cuda")
        bw = torch.full((V, D + pad + offset), 7.0, dtype=torch.float16, device="cuda")
        st = binding.tg_linear_cross_entropy_f16(
            x.data_ptr(), w.data_ptr(), target.data_ptr(), IGNORE, 1.0, dloss.data_ptr(),
            loss.data_ptr(), 0, bx.data_ptr() + 2 * offset, bw.data_ptr() + 2 * offset, T, V, D, x.stride(0),
            w.stride(0), bx.stride(0), bw.stride(0), None,
            torch.cuda.current_stream().cuda_stream)
        assert st == binding.TG_OK
        # the plan, and with it the order of a sum, may go by the output's alignment
        check(x, w, 0, 1.0, q, live, zero, dloss, loss, None, bx[:, offset:offset + D],
              bw[:, offset:offset + D])
        for buf in (bx, bw):
            assert (buf[:, :offset] == 7).all() and (buf[:, offset + D:] == 7).all()


@pytest.mark.parametrize("which", ["loss", "distil"])
def test_against_differences(which):
    T, V, D = 12, 90, 32
    x, w = operands(T, V, D, 0, 111)
    dloss = torch.rand(T, generator=gen(112), device="cuda") + 0.5
    if which == "loss":
        target = targets(T, V, 113, 0.1)
        q, live = one_hot(target, V)
        entropy, tau = torch.zeros(T, dtype=D64, device="cuda"), 1.0
        _, dx, dw = tg.linear_cross_entropy_step(x, w, target, dloss)
    else:
        index, logits = teacher(T, V, 7, 114, torch.float32)
        tau = 2.0
        q, live, entropy = teacher_q(index, logits, tau, V)
        _, dx, dw = tg.linear_distillation_step(x, w, index, logits, dloss, temperature=tau)

    def total(xd, wd):
        z = xd @ wd.t() / tau
        each = entropy + torch.logsumexp(z, 1) - (q * z).sum(1)
        return (dloss.to(D64) * torch.where(live, each, torch.zeros_like(each))).sum()

    args = [x.to(D64), w.to(D64)]
    for k, grad in enumerate((dx, dw)):
        way = torch.randn(args[k].shape, generator=gen(115), device="cuda", dtype=D64)
        up, down = list(args), list(args)
        up[k], down[k] = args[k] + 1e-5 * way, args[k] - 1e-5 * way
        diff = (total(*up) - total(*down)) / 2e-5
        got = (grad.to(D64) * way).sum()
        # per element: G's rounding (2^-11 of terms that mostly add up) and the output's, within
        # 2^-8 of the element's size or the largest's 2^-10
        mag = grad.to(D64).abs()
        assert (got - diff).abs() <= ((mag * 2 ** -8 + mag.max() * 2 ** -10) * way.abs()).sum()


def test_other_stream_and_threads():
    import threading

    T, V, D = 200, 5000, 256
    x, w = operands(T, V, D, 0, 116)
    target = targets(T, V, 117)
    dloss = torch.ones(T, device="cuda")
    want = tg.linear_cross_entropy_step(x, w, target, dloss)
    torch.cuda.synchronize()
    got = {}

    def work(k):
        s = torch.cuda.Stream()
        for _ in range(5):
            got[k] = tg.linear_cross_entropy_step(x, w, target, dloss, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4
    for g in got.values():
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_calls_back_to_back():
    """Calls that share scratch and follow one another without a wait give what they give alone."""
    calls = []
    for k, (T, V, D, layout) in enumerate([
            (1, 5000, 256, tg.TG_HEAD_VOCAB_MAJOR), (130, 3000, 136, tg.TG_HEAD_WIDTH_MAJOR),
            (600, 2000, 64, tg.TG_HEAD_VOCAB_MAJOR), (16, 40000, 1024, tg.TG_HEAD_VOCAB_MAJOR),
            (300, 1001, 77, tg.TG_HEAD_VOCAB_MAJOR)]):
        x, w = operands(T, V, D, layout, 130 + k)
        target, (index, logits) = targets(T, V, 140 + k), teacher(T, V, 9, 150 + k, torch.float16)
        dloss = torch.rand(T, generator=gen(160 + k), device="cuda")
        piece = 256 if T > 256 else 0
        calls += [lambda x=x, w=w, t=target, n=layout: [tg.linear_cross_entropy(x, w, t, layout=n)],
                  lambda x=x, w=w, t=target, d=dloss, n=layout, p=piece:
                      tg.linear_cross_entropy_step(x, w, t, d, layout=n, piece_rows=p),
                  lambda x=x, w=w, i=index, u=logits, n=layout:
                      [tg.linear_distillation(x, w, i, u, 2.0, layout=n)],
                  lambda x=x, w=w, i=index, u=logits, d=dloss, n=layout, p=piece:
                      tg.linear_distillation_step(x, w, i, u, d, 2.0, layout=n, piece_rows=p)]
    want = []
    for c in calls:
        torch.cuda.synchronize()
        want.append(c())
    torch.cuda.synchronize()
    got = [[c() for c in calls] for _ in range(20)]
    torch.cuda.synchronize()
    for run in got:
        for g, e in zip(run, want):
            assert all(torch.equal(a, b) for a, b in zip(g, e))


def test_few_tokens_over_a_large_head():
    """Sizes at which dX and dW run side by side: against the definition, alone, from several threads
    on streams of their own, and captured."""
    import threading

    T, V, D = 9, 26000, 520
    layout = tg.TG_HEAD_VOCAB_MAJOR
    x, w = operands(T, V, D, layout, 170)
    target = targets(T, V, 171)
    dloss = torch.rand(T, generator=gen(172), device="cuda") + 0.5
    want = tg.linear_cross_entropy_step(x, w, target, dloss)
    q, live = one_hot(target, V)
    zero = torch.zeros(T, dtype=D64, device="cuda")
    check(x, w, layout, 1.0, q, live, zero, dloss, want[0], None, *want[1:])
    for layout2 in (layout, tg.TG_HEAD_WIDTH_MAJOR):
        w2 = w if layout2 == layout else rows(w.t())
        got = tg.linear_cross_entropy_step(x, w2, target, dloss, layout=layout2)
        check(x, w2, layout2, 1.0, q, live, zero, dloss, got[0], None, *got[1:])
    torch.cuda.synchronize()
    got = {}

    def work(k):
        s = torch.cuda.Stream()
        for _ in range(5):
            got[k] = tg.linear_cross_entropy_step(x, w, target, dloss, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4
    for g in got.values():
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = tg.linear_cross_entropy_step(x, w, target, dloss)
    graph.replay()
    check(x, w, layout, 1.0, q, live, zero, dloss, inside[0], None, *inside[1:])


def test_graph_capture():
    T, V, D = 130, 2000, 136
    x, w = operands(T, V, D, 0, 118)
    index, logits = teacher(T, V, 8, 119, torch.float16)
    target = targets(T, V, 120)
    dloss = torch.ones(T, device="cuda")
    gamma = torch.ones(D, dtype=torch.float16, device="cuda")

    def work():
        y, mean, rstd = tg.layer_norm(x, gamma, stats=True)
        loss, dy, dw = tg.linear_cross_entropy_step(y, w, target, dloss)
        return (loss, dw, *tg.layer_norm_backward(dy, x, mean, rstd, gamma)[:2],
                *tg.linear_distillation_step(y, w, index, logits, dloss))

    want = work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_timeout_is_reported_and_survived():
    T, V, D = 300, 1000, 256
    x, w = operands(T, V, D, 0, 121)
    target = targets(T, V, 122)
    want = tg.linear_cross_entropy(x, w, target)
    loss = torch.empty(T, device="cuda")
    o = binding.tg_head_options(debug_flags=binding.TG_DEBUG_DROP_FIRST_STAGE, timeout_ms=50)
    st = binding.tg_linear_cross_entropy_f16(
        x.data_ptr(), w.data_ptr(), target.data_ptr(), IGNORE, 1.0, 0, loss.data_ptr(), 0, 0, 0, T,
        V, D, D, D, 0, 0, o, torch.cuda.current_stream().cuda_stream)
    assert st == binding.TG_OK
    st, word = binding.tg_device_error_check(clear=True)
    assert st == binding.TG_ERR_TIMEOUT and word & 1
    assert torch.equal(tg.linear_cross_entropy(x, w, target), want)


def test_refusals():
    x, w = operands(8, 50, 16, 0, 123)
    target = targets(8, 50, 124)
    dloss = torch.ones(8, device="cuda")
    index, logits = teacher(8, 50, 4, 125, torch.float16)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(x.float(), w, target)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(x, w.float(), target)
    with pytest.raises(TypeError):
        tg.linear_cross_entropy(x, w, target.int())
    with pytest.raises(TypeError):
        tg.linear_cross_entropy_step(x, w, target, dloss.half())
    with pytest.raises(TypeError):
        tg.linear_distillation(x, w, index.int(), logits)
    with pytest.raises(TypeError):
        tg.linear_distillation(x, w, index, logits.double())
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x, w.t(), target)
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x, w, target, layout=tg.TG_HEAD_WIDTH_MAJOR)
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x, w, target, layout=7)
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x, w, target[:7])
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x.cpu(), w, target)
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(x, w, target.cpu())
    with pytest.raises(ValueError):
        tg.linear_cross_entropy_step(x, w, target, dloss[:1].expand(8))
    with pytest.raises(ValueError):
        tg.linear_distillation(x, w, index[:, :3], logits[:, :3])
    with pytest.raises(ValueError):
        tg.linear_distillation(x, w, index, logits[:, :3].contiguous())
    with pytest.raises(ValueError):
        tg.linear_distillation(x, w, index[:, :0].contiguous(), logits[:, :0].contiguous())
    with pytest.raises(tg.TgError):
        tg.linear_cross_entropy(x, w, target, logit_scale=0.0)
    with pytest.raises(tg.TgError):
        tg.linear_distillation(x, w, index, logits, temperature=-1.0)
    with pytest.raises(tg.TgError):
        tg.linear_cross_entropy(x, w, target, piece_rows=-5)
