"""The gated product and its gradients for few tokens over weights large enough that the calls are bound by
reading and writing them: splits chosen by the reading time, dX beside both weights' gradients in one launch.
Tolerances as in test_gpu_gated.py."""

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_gated import (  # noqa: E402,F401
    ACTS, _built, check_backward, check_forward, gen, operands, rows)

SIZES = [(1, 2048, 2304, 0, 0), (7, 4100, 1032, 0, 0), (8, 1031, 4500, 0, 0), (64, 8192, 1024, 0, 0),
         (65, 2500, 2100, 4, 0), (100, 1111, 4444, 3, 1), (128, 20000, 520, 0, 0), (128, 4096, 4096, 8, 8),
         (2, 777, 9000, 1, 3), (33, 30000, 256, 0, 0), (129, 4096, 1024, 0, 0),
         (256, 5000, 2047, 3, 0), (200, 2300, 2304, 0, 0), (257, 4100, 1100, 0, 0)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K,pad,offset", SIZES)
def test_few_tokens(M, N, K, pad, offset, trans):
    x, wg, wu = operands(M, N, K, trans, 60, pad, offset)
    h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
    check_forward(x, wg, wu, trans, "silu", h, gate, up)
    dh = rows(torch.randn(M, N, generator=gen(61), device="cuda") * 0.25, pad, offset)
    got = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
    check_backward(dh, x, wg, wu, gate, up, trans, "silu", *got)
    again = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    dx = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, weight_grads=False)[0]
    dw = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, input_grad=False)
    check_backward(dh, x, wg, wu, gate, up, trans, "silu", dx, *dw[1:])


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", [(64, 4096, 2048), (5, 3000, 1500)])
def test_captured(M, N, K, trans):
    x, wg, wu = operands(M, N, K, trans, 62)
    dh = (torch.randn(M, N, generator=gen(63), device="cuda") * 0.25).half()

    def step():
        h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
        return h, gate, up, *tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("options", [
    dict(block_n=128, pair=-1), dict(block_n=256, pair=-1), dict(pair=1), dict(split_k=3, pair=-1),
    dict(split_k=2, pair=1), dict(split_k=5, block_n=256, pair=-1), dict(max_ctas=4), dict(panel_m=2)])
@pytest.mark.parametrize("M,N,K", [(40, 520, 1000), (600, 392, 712), (261, 1027, 330)])
@pytest.mark.parametrize("trans", [False, True])
def test_plans_of_the_backward_pass(M, N, K, trans, options):
    x, wg, wu = operands(M, N, K, trans, 64)
    _, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
    dh = (torch.randn(M, N, generator=gen(65), device="cuda") * 0.25).half()
    check_backward(dh, x, wg, wu, gate, up, trans, "silu",
                   *tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans, options=options))


@pytest.mark.parametrize("M,N,K", [(2, 64, 40000), (40000, 72, 40), (130, 100, 33000)])
def test_long_sums(M, N, K):
    """Sums of more terms than one accumulator takes: the width forward, the tokens in dW."""
    x, wg, wu = operands(M, N, K, False, 66)
    h, gate, up = tg.gated_linear(x, wg, wu, keep=True)
    check_forward(x, wg, wu, False, "silu", h, gate, up)
    dh = (torch.randn(M, N, generator=gen(67), device="cuda") * 0.25).half()
    check_backward(dh, x, wg, wu, gate, up, False, "silu",
                   *tg.gated_linear_backward(dh, x, wg, wu, gate, up))


@pytest.mark.parametrize("K,N", [(8192, 64), (28672, 512), (4096, 1000), (1024, 256), (16384, 136)])
@pytest.mark.parametrize("M", [1, 5, 64, 128])
def test_narrow_weights(M, K, N):
    """Few tiles of a long sum: split."""
    for trans in (False, True):
        x, wg, wu = operands(M, N, K, trans, 85)
        h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
        check_forward(x, wg, wu, trans, "silu", h, gate, up)


def test_rows_of_nan_stay_apart():
    """Few tokens' operands lie in scratch of eight rows: what is behind them does not come in, and a row of
    NaN spoils its own dx alone."""
    M, N, K = 3, 2048, 2304
    x, wg, wu = operands(M, N, K, False, 68)
    for _ in range(3):  # the pool's memory is full of NaN
        junk = torch.full((64, 8192), float("nan"), dtype=torch.float16, device="cuda")
        tg.gated_linear(junk[:, :K], wg, wu)
    _, gate, up = tg.gated_linear(x, wg, wu, keep=True)
    dh = (torch.randn(M, N, generator=gen(69), device="cuda") * 0.25).half()
    want = tg.gated_linear_backward(dh, x, wg, wu, gate, up)
    check_backward(dh, x, wg, wu, gate, up, False, "silu", *want)
    bad = dh.clone()
    bad[1] = float("nan")
    dx, dwg, _ = tg.gated_linear_backward(bad, x, wg, wu, gate, up)
    assert dx[1].isnan().all() and torch.equal(dx[0], want[0][0]) and torch.equal(dx[2], want[0][2])
    assert dwg.isnan().all()


def test_a_wait_that_runs_out():
    M, N, K = 64, 4096, 2048
    x, wg, wu = operands(M, N, K, False, 70)
    h, gate, up = tg.gated_linear(x, wg, wu, keep=True)
    want = tg.gated_linear_backward(h, x, wg, wu, gate, up)
    options = dict(debug_flags=binding.TG_DEBUG_DROP_FIRST_STAGE, timeout_ms=20)
    tg.gated_linear_backward(h, x, wg, wu, gate, up, options=options)
    st, word = binding.tg_device_error_check(clear=True)
    assert st == binding.TG_ERR_TIMEOUT and word & 1
    assert all(torch.equal(a, b) for a, b in zip(want, tg.gated_linear_backward(h, x, wg, wu, gate, up)))
    assert binding.tg_device_error_check(clear=True)[0] == binding.TG_OK
