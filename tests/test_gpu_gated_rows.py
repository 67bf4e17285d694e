"""The gated product of up to four tokens over weights whose rows start anywhere, read where they are.
Tolerances as in test_gpu_gated.py; what lies beside a row, a gap or another allocation's end, is NaN."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_gated import ACTS, _built, check_forward, gen  # noqa: E402,F401


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
    want = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
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
