"""The gated product of up to four tokens over weights whose rows start anywhere, read where they are.
Tolerances as in test_gpu_gated.py; what lies beside a row, a gap or another allocation's end, is NaN."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_gated import ACTS, _built, check_backward, check_forward, gen  # noqa: E402,F401


def between_nan(t, pad, offset):
    """t's values in rows of a buffer that is NaN everywhere else, from its element `offset` on; a pad of -1: rows
    without a gap."""
    m, n = t.shape
    ld = n + max(pad, 0)
    buf = torch.full((offset + m * ld + 16,), math.nan, dtype=torch.float16, device="cuda")
    view = buf.as_strided((m, n), (ld, 1), offset)
    view.copy_(t)
    return view


def operands(M, N, K, trans, seed, pad, offsets):
    g = gen(seed)
    x = between_nan(torch.randn(M, K, generator=g, device="cuda"), pad, offsets[2])
    ws = []
    for o in offsets[:2]:
        w = torch.randn(K, N, generator=g, device="cuda") * (1.5 / math.sqrt(K))
        ws.append(between_nan(w.t() if trans else w, pad, o))
    return x, *ws


SIZES = [(1, 1), (1, 5), (5, 1), (2, 2), (7, 3), (126, 8), (127, 63), (128, 64), (125, 65), (129, 257), (253, 1024),
         (252, 1025), (257, 2047), (64, 2048), (33, 2049), (1000, 1031), (4097, 515), (515, 4097), (3, 9001),
         (9001, 3), (2051, 2305)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", SIZES)
def test_sizes(M, N, K, trans):
    for pad, offsets in ((0, (1, 0, 0)), (1, (0, 3, 1)), (2, (1, 1, 5)), (0, (2, 4, 3))):
        x, wg, wu = operands(M, N, K, trans, N + K, pad, offsets)
        h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
        check_forward(x, wg, wu, trans, "silu", h, gate, up)
        assert torch.equal(h, tg.gated_linear(x, wg, wu, trans_w=trans))


def pre_activations(M, N, seed, pad, offset):
    g = gen(seed)
    return [between_nan(torch.randn(M, N, generator=g, device="cuda") * s, pad, offset) for s in (0.25, 1.5, 1.5)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 2051, 1031), (2, 2305, 2051), (3, 4097, 2053), (4, 2053, 4097), (4, 515, 16389),
                                   (3, 16389, 515), (2, 5, 1000001), (2, 1000001, 5), (1, 1, 2100001), (1, 2100001, 1),
                                   (4, 127, 66053), (4, 66053, 127), (1, 1024, 2049), (2, 2048, 2049), (1, 2049, 1024)])
def test_gradients(M, N, K, trans):
    for pad, offsets in ((0, (1, 0, 0)), (1, (0, 3, 1)), (0, (2, 4, 3))):
        x, wg, wu = operands(M, N, K, trans, N + K, pad, offsets)
        dh, gate, up = pre_activations(M, N, 86, pad, offsets[1])
        got = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
        check_backward(dh, x, wg, wu, gate, up, trans, "silu", *got)
        dx = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, weight_grads=False)[0]
        dw = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, input_grad=False)[1:]
        assert all(torch.equal(a, b) for a, b in zip(got, (dx, *dw)))


def test_gradients_of_very_many_rows():
    M, N, K = 1, 3, 65535 * 128 + 130
    x, wg, wu = operands(M, N, K, False, 87, 0, (1, 0, 0))
    dh, gate, up = pre_activations(M, N, 88, 0, 0)
    check_backward(dh, x, wg, wu, gate, up, False, "silu", *tg.gated_linear_backward(dh, x, wg, wu, gate, up))


def test_gradients_into_views():
    """One weight's gradient alone, rows that start anywhere and what is beside them."""
    from fp16_gemm_relu_gb300 import binding

    M, N, K, pad = 2, 2305, 2051, 3
    x, wg, wu = operands(M, N, K, False, 89, 1, (1, 2, 0))
    dh, gate, up = pre_activations(M, N, 90, 0, 0)
    want = tg.gated_linear_backward(dh, x, wg, wu, gate, up)
    stream = torch.cuda.current_stream().cuda_stream
    for which in ((1, 0), (0, 1), (1, 1)):
        for offset in (0, 1):
            bufs = [torch.full((K * (N + pad) + 8,), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
            views = [b.as_strided((K, N), (N + pad, 1), offset) for b in bufs]
            st = binding.tg_gated_backward_f16(
                dh.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), gate.data_ptr(), up.data_ptr(), 0,
                *(v.data_ptr() if w else 0 for v, w in zip(views, which)), binding.TG_ACT_SILU, 0, M, N, K, N,
                x.stride(0), wg.stride(0), wu.stride(0), N, N, 0, N + pad, N + pad, stream=stream)
            assert st == binding.TG_OK
            for b, v, w, ref in zip(bufs, views, which, want[1:]):
                if w:
                    assert torch.equal(v, ref)
                    v.fill_(9.0)
                assert (b == 9).all()


@pytest.mark.parametrize("trans", [False, True])
def test_gradients_of_rows_of_nan(trans):
    M, N, K = 3, 4097, 2053
    x, wg, wu = operands(M, N, K, trans, 91, 0, (1, 0, 1))
    dh, gate, up = pre_activations(M, N, 92, 0, 1)
    want = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
    bad = dh.clone()
    bad[1] = math.nan
    dx, dwg, dwu = tg.gated_linear_backward(bad, x, wg, wu, gate, up, trans_w=trans)
    assert dx[1].isnan().all() and torch.equal(dx[::2], want[0][::2]) and dwg.isnan().all() and dwu.isnan().all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("act", list(ACTS))
def test_activations_and_outputs(act, trans):
    """Rows of the output that start anywhere; what is beside them stays."""
    M, N, K = 3, 333, 1111
    x, wg, wu = operands(M, N, K, trans, 80, 3, (1, 2, 0))
    buf = torch.full((M, N + 5), 9.0, dtype=torch.float16, device="cuda")
    h = tg.gated_linear(x, wg, wu, ACTS[act], trans_w=trans, out=buf[:, 3:3 + N])
    check_forward(x, wg, wu, trans, act, h)
    assert (buf[:, :3] == 9).all() and (buf[:, 3 + N:] == 9).all()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 300, 5000), (4, 5000, 300)])
def test_tokens_do_not_meet(M, N, K, trans):
    """A token that is not finite spoils its own outputs alone, and an infinite element at a sum's end gives what its
    weight makes of it."""
    x, wg, wu = operands(4, N, K, trans, 81, 0, (1, 1, 1))
    want = tg.gated_linear(x, wg, wu, trans_w=trans)
    bad = x.clone()
    bad[1], bad[3] = math.nan, math.inf
    got = tg.gated_linear(bad, wg, wu, trans_w=trans)
    assert torch.equal(got[::2], want[::2]) and got[1].isnan().all()
    for at in (0, K - 1):
        one = x[:1].clone()
        one[0, at] = math.inf
        _, gate, _ = tg.gated_linear(one, wg, wu, trans_w=trans, keep=True)
        w = (wg[:, at] if trans else wg[at]).float()
        assert torch.equal(gate[0].float()[w != 0], w[w != 0].sign() * math.inf)


def test_extreme_weights():
    """A column (a row) of NaN is that output's alone."""
    M, N, K = 2, 400, 700
    for trans in (False, True):
        x, wg, wu = operands(M, N, K, trans, 82, 0, (1, 0, 0))
        want = tg.gated_linear(x, wg, wu, trans_w=trans)
        for n in (0, 125, 126, 127, 252, N - 1):
            bad = between_nan(wg.clone(), 0, 1)
            (bad[n] if trans else bad[:, n]).fill_(math.nan)
            got = tg.gated_linear(x, bad, wu, trans_w=trans)
            keep = torch.arange(N, device="cuda") != n
            assert got[:, n].isnan().all() and torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("trans", [False, True])
def test_same_bits_captured_and_on_a_stream(trans):
    M, N, K = 2, 3001, 2999
    x, wg, wu = operands(M, N, K, trans, 83, 0, (0, 1, 0))

    def step(stream=None):
        h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True, stream=stream)
        return h, gate, up, *tg.gated_linear_backward(h, x, wg, wu, gate, up, trans_w=trans, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, got):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("trans", [False, True])
def test_long_offsets(trans):
    """Weights of more than 2^31 elements: the row's offset in 64 bits."""
    M, N, K = 1, 46349, 46351
    g = gen(84)
    x = torch.randn(M, K, generator=g, device="cuda").half()
    w = torch.empty((N, K) if trans else (K, N), dtype=torch.float16, device="cuda")
    for i in range(0, w.shape[0], 4096):
        w[i:i + 4096] = torch.randn(w[i:i + 4096].shape, generator=g, device="cuda") / 128
    h, gate, up = tg.gated_linear(x, w, w, trans_w=trans, keep=True)
    at = torch.tensor([0, 1, 125, 126, 20000, N - 2, N - 1], device="cuda")
    part = (w[at] if trans else w[:, at]).contiguous()
    check_forward(x, part, part, trans, "silu", h[:, at], gate[:, at], up[:, at])
