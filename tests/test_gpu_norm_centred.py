"""Layer norm's backward pass of rows whose mean is far larger than their spread, and of gradients that
follow the normalised row, which dx cancels: against the definition in 64 bits.

Tolerances: those of tests/test_gpu_norm.py (check_backward).  Centred arithmetic stays within 2^-16 of
rstd (|g| + mean|g| + |h| mean|g h|): x - mean is one rounding, and the sums are within 2^-18.6 of their
sums of magnitudes.  Uncentred, a row would be off by up to 2^-24 |mean| / spread of |h| mean|g h| (2^-13
at 2000 spreads)."""

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_norm import EPS, _built, check_backward, make  # noqa: E402,F401

WIDTHS = [(64, 512), (64, 513), (64, 1000), (64, 4096), (33, 4099), (33, 8192), (33, 8200), (17, 12001),
          (17, 16384), (17, 16385), (17, 20000)]


@pytest.mark.parametrize("M,N", WIDTHS)
@pytest.mark.parametrize("shift,spread", [(100.0, 0.1), (1000.0, 0.5), (-1000.0, 0.5)])
@pytest.mark.parametrize("along,noise", [(0.7, 0.7), (1.0, 0.0)])
def test_far_from_zero(M, N, shift, spread, along, noise):
    x = make(M, N, seed=80, scale=spread, shift=shift)
    gamma = torch.ones(N, dtype=torch.float16, device="cuda")
    _, mean, rstd = tg.layer_norm(x, gamma, eps=EPS, stats=True)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    dy = (along * h + noise * make(M, N, seed=81).double()).half()
    check_backward(dy, x, gamma, mean, rstd, *tg.layer_norm_backward(dy, x, mean, rstd, gamma))


@pytest.mark.parametrize("N", [512, 1000, 4096, 9000, 20000])
def test_constant_rows_and_a_tiny_eps(N):
    """rstd = 1 / sqrt(eps) of a row without spread: 1e15 here, whose cube is no float32."""
    x = torch.full((5, N), 2.0, dtype=torch.float16, device="cuda")  # its mean is exact
    _, mean, rstd = tg.layer_norm(x, eps=1e-30, stats=True)
    assert (mean == 2).all()
    dx, dgamma, dbeta = tg.layer_norm_backward(torch.zeros_like(x), x, mean, rstd)
    assert (dx == 0).all() and (dgamma == 0).all() and (dbeta == 0).all()
