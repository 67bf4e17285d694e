"""The gated product and its gradients where a matrix has more than 2^31 elements: offsets in 64 bits, on rows that TMA
stores and on rows that start anywhere.

Compared are the first and the last rows of h, the pre-activations and dX, with the tolerances of test_gpu_gated.py, and
the weights' gradients whole, as root mean squares: dG and the result are rounded to fp16, each by at most
2^-11 and as a root mean square by 2^-11 / sqrt(3), together less than 2^-11.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_gated import D64, _built, act64, check_backward, check_forward, gen, operands  # noqa: E402,F401


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", [(131200, 16400, 24), (135001, 16385, 9)])
def test_more_than_2_31_elements(M, N, K, trans):
    assert M * N > 2 ** 31
    x, wg, wu = operands(M, N, K, trans, 1)
    h, gate, up = tg.gated_linear(x, wg, wu, trans_w=trans, keep=True)
    for rows in (slice(0, 300), slice(M - 300, M)):
        check_forward(x[rows], wg, wu, trans, "silu", h[rows], gate[rows], up[rows])
    assert torch.equal(tg.gated_linear(x[M // 2:], wg, wu, trans_w=trans), h[M // 2:])
    dh = h.normal_(generator=gen(2)).mul_(0.25)
    dx, dwg, dwu = tg.gated_linear_backward(dh, x, wg, wu, gate, up, trans_w=trans)
    for rows in (slice(0, 300), slice(M - 300, M)):
        check_backward(dh[rows], x[rows], wg, wu, gate[rows], up[rows], trans, "silu", dx[rows], None, None)
    refs = [torch.zeros(K, N, dtype=D64, device="cuda") for _ in range(2)]
    for a in range(0, M, 4096):
        rows = slice(a, min(a + 4096, M))
        value, slope = act64(gate[rows].to(D64), "silu")
        d, xt = dh[rows].to(D64), x[rows].to(D64).t()
        refs[0] += xt @ (d * up[rows].to(D64) * slope)
        refs[1] += xt @ (d * value)
    for got, ref in zip((dwg, dwu), refs):
        off = (got.t() if trans else got).to(D64) - ref
        assert float(off.norm()) <= 2 ** -11 * float(ref.norm()) and got.shape == wg.shape
