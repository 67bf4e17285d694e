"""How exact the sum of squares of the gradients' norm is.

A thread adds the 32 squares of a chunk in four sums of eight, each step within 2^-24 of its sum, meets them in two
more, and adds chunks with what is rounded off carried along (2 * 2^-24 in all, and a step that takes it off); a warp's
sums meet in five steps, a block's eight in seven, the blocks' in float64.  25 steps: within 25 * 2^-24 of the sum of
squares, half of that for the norm, and its rounding to float32: 14 * 2^-24, 8.3e-7, at the very worst.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from tests.test_gpu_head import D64, _built, gen  # noqa: E402,F401

WORST = 14 * 2 ** -24


def norm64(t):
    return math.sqrt(sum(float(p.to(D64).square().sum()) for p in t.split(1 << 26)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("n", [8191, 3000 * 4099, (1 << 28) + 12345])
def test_random(n, dtype):
    g = torch.empty(n, dtype=dtype, device="cuda")
    for i in range(0, n, 1 << 26):
        part = g[i:i + (1 << 26)]
        part.copy_(torch.randn(part.shape, generator=gen(1 + i), device="cuda"))
    ref = norm64(g)
    for scale in (1.0, 8192.0):
        assert abs(float(tg.gradient_norm([g], scale)) * scale - ref) <= WORST * ref


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_small_squares_after_large_ones(dtype):
    """Every thread's sum begins with 2^21 or more and then meets 0.125 again and again, half a unit of its last place
    or less: added up without the carried remainder they are lost, 3.8e-6 of the norm."""
    n, large = 1 << 30, 1 << 23  # (a thread's first chunks: there are fewer blocks than 1024 chunks)
    g = torch.full((n,), 2.0 ** -4, dtype=dtype, device="cuda")
    g[:large] = 256.0
    ref = math.sqrt(large * 65536.0 + (n - large) / 256.0)
    lost = 1 - math.sqrt(large * 65536.0) / ref
    assert lost > 2 * WORST
    norm = float(tg.gradient_norm([g]))
    assert abs(norm - ref) <= WORST * ref
