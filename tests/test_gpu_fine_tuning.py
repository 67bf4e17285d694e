"""A fine-tuning step as it is used: a gated block with its residual, a layer norm, and a preference or policy
loss of the head, their backward passes, and the gradients unscaled and clipped.

Tolerance.  Every value that passes from one operator to the next is fp16, rounded by at most 2^-11 of itself; a
gradient has come through at most ten of them (h, its residual, the norm, G, dX, dX of the norm, the kept
pre-activations, dG and dU, and itself), whose errors are independent of each other and of the data: as root
mean squares over a tensor at most sqrt(10) 2^-11 / sqrt(3) < 2^-10 of its size each way, and twice that where
two such paths meet (the gradient of the residual's input).  The loss's own derivative is smooth.  2^-8 bounds both.
"""

import math
import threading

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402
from tests.test_gpu_head import D64, IGNORE, _built, gen  # noqa: E402,F401

T, D, H, V, PAIRS = 192, 136, 264, 1000, 4
SCALE = 256.0


def model(seed=1):
    g = gen(seed)

    def normal(*shape, size):
        return (torch.randn(*shape, generator=g, device="cuda") * size).half()

    x = normal(T, D, size=1.0)
    weights = {"gate": normal(D, H, size=D ** -0.5), "up": normal(D, H, size=D ** -0.5),
               "down": normal(H, D, size=H ** -0.5), "gamma": 1 + normal(D, size=0.1),
               "beta": normal(D, size=0.1), "head": normal(V, D, size=2 * D ** -0.5)}
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::9] = IGNORE
    offsets = torch.tensor([0, 20, 50, 60, 60, 100, 140, 170, 185], device="cuda")
    reference = -math.log(V) + torch.randn(T, generator=g, device="cuda")
    return x, weights, target, offsets, reference


def project(h, w):
    """h @ w with the framework's GEMM, its backward by the framework's transposed ones."""
    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, b):
            ctx.save_for_backward(a, b)
            return tg.gemm_relu(a, b, epilogue=tg.TG_EPILOGUE_NONE)

        @staticmethod
        def backward(ctx, d):
            a, b = ctx.saved_tensors
            return autograd.gemm_t(d, b, 0, 1), autograd.gemm_t(a, d, 1, 0)

    return Product.apply(h, w)


def losses64(x, w, target, offsets, reference, old, advantage):
    f = torch.nn.functional
    h = f.silu(x @ w["gate"]) * (x @ w["up"])
    y = f.layer_norm(x + h @ w["down"], (D,), w["gamma"], w["beta"])
    live = target != IGNORE
    logp = torch.log_softmax(y @ w["head"].t(), 1).gather(1, target.clamp_min(0)[:, None])[:, 0] * live
    d = (logp - reference.to(D64)) * live
    at = offsets.tolist()
    sums = torch.stack([d[a:b].sum() for a, b in zip(at[:-1], at[1:])]).view(-1, 2)
    preference = -f.logsigmoid(0.2 * (sums[:, 0] - sums[:, 1])).mean()
    ratio = torch.exp(logp - old.to(D64))
    a = advantage.to(D64)
    away = reference.to(D64) - logp
    each = -torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) + 0.01 * (torch.exp(away) - away - 1)
    return preference, (each * live).sum() / live.sum(), logp


@pytest.mark.parametrize("which", ["preference", "policy"])
def test_step(which):
    x, w, target, offsets, reference = model()
    live = target != IGNORE
    with torch.no_grad():
        _, _, logp = losses64(x.to(D64), {k: v.to(D64) for k, v in w.items()}, target, offsets, reference,
                              reference, reference)
    moved = 0.5 * torch.randn(T, generator=gen(2), device="cuda", dtype=D64)
    for border in (math.log(0.8), math.log(1.2)):  # off the clipping's borders by more than fp16 moves logp
        moved = torch.where((moved - border).abs() < 0.06, moved + 0.13, moved)
    old = (logp - moved).float()
    advantage = torch.randn(T, generator=gen(3), device="cuda")

    leaves = {k: v.clone().requires_grad_(True) for k, v in w.items()}
    xin = x.clone().requires_grad_(True)
    h = autograd.gated_linear(xin, leaves["gate"], leaves["up"])
    y = autograd.layer_norm(xin + project(h, leaves["down"]), leaves["gamma"], leaves["beta"])
    if which == "preference":
        loss, _ = autograd.linear_preference(y, leaves["head"], target, offsets, reference, beta=0.2)
    else:
        loss, _ = autograd.linear_policy(y, leaves["head"], target, old, advantage, reference, kl_weight=0.01)
    (loss * SCALE).backward()
    names = list(leaves)
    scaled = [leaves[k].grad for k in names]
    norm, grads = tg.clip_gradients(scaled, 1e9, SCALE)
    half, clipped = tg.clip_gradients(scaled, float(norm) / 2, SCALE)

    ref = {k: v.to(D64).requires_grad_(True) for k, v in w.items()}
    xr = x.to(D64).requires_grad_(True)
    preference, policy, _ = losses64(xr, ref, target, offsets, reference, old, advantage)
    want = preference if which == "preference" else policy
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 2 ** -8 * (abs(float(want.detach())) + 1)
    total = math.sqrt(sum(float(r.grad.square().sum()) for r in ref.values()))
    assert abs(float(norm) - total) <= 2 ** -8 * total and torch.equal(norm, half)
    for k, g, c in zip(names, grads, clipped):
        r = ref[k].grad
        assert float((g.to(D64) - r).norm()) <= 2 ** -8 * float(r.norm()), k
        assert float((c.to(D64) - r / 2).norm()) <= 2 ** -8 * float(r.norm()), k
    assert float((xin.grad.to(D64) / SCALE - xr.grad).norm()) <= 2 ** -8 * float(xr.grad.norm())
    assert live.any()


def step(x, w, target, offsets, reference, dloss, stream=None):
    """The same without autograd: everything that the step gives."""
    h, gate, up = tg.gated_linear(x, w["gate"], w["up"], keep=True, stream=stream)
    y, mean, rstd = tg.layer_norm(x, w["gamma"], w["beta"], stats=True, stream=stream)
    loss, ratios, dy, dhead = tg.linear_preference_step(y, w["head"], target, offsets, dloss, reference,
                                                        stream=stream)
    dx, dgamma, dbeta = tg.layer_norm_backward(dy, x, mean, rstd, w["gamma"], stream=stream)
    dx2, dgate, dup = tg.gated_linear_backward(h, x, w["gate"], w["up"], gate, up, stream=stream)
    norm, grads = tg.clip_gradients([dhead, dgamma, dbeta, dgate, dup], 1.0, SCALE, stream=stream)
    return [h, gate, up, loss, ratios, dx, dx2, norm, *grads]


def test_two_graphs_at_once():
    """Two captured steps replayed side by side on two streams, again and again, with eager calls between."""
    x, w, target, offsets, reference = model(4)
    x2, w2 = model(5)[:2]
    dloss = torch.full((PAIRS,), SCALE / PAIRS, device="cuda")
    want = [step(a, b, target, offsets, reference, dloss) for a, b in ((x, w), (x2, w2))]
    torch.cuda.synchronize()
    graphs, got = [], []
    for a, b in ((x, w), (x2, w2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(a, b, target, offsets, reference, dloss))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for r in got:
            for t in r:
                t.fill_(-1.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        again = step(x, w, target, offsets, reference, dloss)
        torch.cuda.synchronize()
        for a, b in zip(want + [want[0]], got + [again]):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_many_threads():
    """Steps from several host threads on streams of their own give the same bits."""
    data = [model(6 + i) for i in range(4)]
    dloss = torch.full((PAIRS,), SCALE / PAIRS, device="cuda")
    want = [step(*d[:2], *d[2:], dloss) for d in data]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(15):
                got[i] = step(*data[i][:2], *data[i][2:], dloss, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_time_limit():
    """A wait that runs out (the first stage is never filled) ends the call with the error word set, and the
    next call is as ever."""
    x, w = model(10)[:2]
    want = tg.gated_linear(x, w["gate"], w["up"], keep=True)
    fault = dict(debug_flags=binding.TG_DEBUG_DROP_FIRST_STAGE, timeout_ms=20)
    calls = [lambda o: tg.gated_linear(x, w["gate"], w["up"], options=dict(fault, **o)),
             lambda o: tg.gated_linear_backward(want[0], x, w["gate"], w["up"], *want[1:],
                                                options=dict(fault, **o))]
    for call in calls:
        for plan in (dict(pair=1), dict(pair=-1, block_n=256), dict(pair=-1, block_n=128), dict(pair=-1, split_k=2)):
            call(plan)
            st, word = binding.tg_device_error_check(clear=True)
            assert st == binding.TG_ERR_TIMEOUT and word & 1
    again = tg.gated_linear(x, w["gate"], w["up"], keep=True)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    assert binding.tg_device_error_check(clear=True)[0] == binding.TG_OK


def test_example_runs():
    import importlib.util
    import os

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("tune_preference",
                                                  os.path.join(root, "examples", "tune_preference.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    seen = mod.run(steps=3, pairs=4, length=16, width=128, hidden=256, vocab=500, quiet=True)
    assert len(seen) == 3 and all(math.isfinite(v) for row in seen for v in row)
