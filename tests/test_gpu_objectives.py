"""Preference and policy losses of a linear head on the GPU, with their gradients, against the formulas in
64 bits.

Tolerances.  A target's log probability is within e = 2 dz + 2^-19 (|lse| + |z| + 1), dz the bound of a
float32 logit (test_gpu_head.py says why).  A ratio adds up its rows' e and is rounded once; with the
margin m off by em = beta (both ratios' errors) + 2^-22 |m|, the loss is off by at most em (its slope is at
most 1) and 2^-20 of itself and 1; a row's weight beta (sigma(-m) - smoothing) dloss by beta |dloss| (em / 4 +
2^-20).  A policy's ratio r is within r (e + 2^-20), its loss within |A| times that, the penalty's within
|e^d - 1| e + 2^-20 (e^d + |d| + 1), the slopes likewise.  The inputs keep off the clipping's borders.  An
error dw of a row's weight adds dw |p - q| to its row of G; the rest is as for cross entropy.
"""

import math

import pytest

from fp16_gemm_relu_gb300 import binding

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import fp16_gemm_relu_gb300 as tg  # noqa: E402
from fp16_gemm_relu_gb300 import autograd  # noqa: E402
from tests.test_gpu_head import D64, IGNORE, _built, gen, operands, targets  # noqa: E402,F401

VOCAB, WIDTH = tg.TG_HEAD_VOCAB_MAJOR, tg.TG_HEAD_WIDTH_MAJOR


class Head:
    """Logits, log probabilities and their error bounds in 64 bits."""

    def __init__(self, x, w, target, layout, scale=1.0):
        self.w = (w if layout == VOCAB else w.t()).to(D64)
        self.x, self.layout, self.scale = x.to(D64), layout, scale
        D = self.x.shape[1]
        z = scale * self.x @ self.w.t()
        self.dz = scale * D * 2 ** -23 * (self.x.abs() @ self.w.abs().t())
        lse = torch.logsumexp(z, 1)
        self.p = torch.exp(z - lse[:, None])
        self.live = target != IGNORE
        at = target.clamp_min(0)[:, None]
        zt = z.gather(1, at)[:, 0]
        zero = torch.zeros_like(lse)
        self.logp = torch.where(self.live, zt - lse, zero)
        self.e = torch.where(self.live, 2 * self.dz.amax(1) + 2 ** -19 * (lse.abs() + zt.abs() + 1), zero)
        self.q = torch.zeros_like(z).scatter_(1, at, self.live[:, None].to(D64))

    def check_grads(self, w, dw, dx, dweight):
        """w: the rows' weights (of the cross entropy), dw: how far off they may be."""
        w, dw = (torch.where(self.live, t, torch.zeros_like(t))[:, None] for t in (w, dw))
        pq = self.p - self.q
        size = w.abs() + dw
        G = w * pq
        dG = (size * (self.p * (2 * self.dz + 2 ** -18) + 2 ** -18 * self.q + 2 ** -11 * pq.abs())
              + dw * pq.abs() + size.max() * 2 ** -39)
        dG = self.scale * torch.where(self.live[:, None], dG, torch.zeros_like(dG))
        G = self.scale * G
        T, V = G.shape
        for got, ref, err, n, mag in (
                (dx, G @ self.w, dG @ self.w.abs(), V, G.abs() @ self.w.abs()),
                (dweight if self.layout == VOCAB else dweight.t(), G.t() @ self.x,
                 dG.t() @ self.x.abs(), T, G.abs().t() @ self.x.abs())):
            tol = err + (n + 8) * 2 ** -23 * mag + 2 ** -11 * ref.abs() + 2 ** -24
            assert got.shape == ref.shape and got.dtype == torch.float16
            bad = ~((got.to(D64) - ref).abs() <= tol)
            assert not bad.any(), (int(bad.sum()), float(((got.to(D64) - ref).abs() - tol).max()))


def pair_reference(head, target, offsets, reference, beta, smooth, average):
    """(loss, its error, ratios, their error, slope of each row's weight, its error) for dloss 1."""
    ref = torch.zeros_like(head.logp) if reference is None else reference.to(D64)
    at = offsets.tolist()
    ratios, errors, counts = [], [], []
    for a, b in zip(at[:-1], at[1:]):
        keep = head.live[a:b]
        n = max(int(keep.sum()), 1) if average else 1
        ratios.append(((head.logp - ref)[a:b] * keep).sum() / n)
        errors.append((head.e[a:b] * keep).sum() / n)
        counts.append(n)
    ratios, errors = torch.stack(ratios).view(-1, 2), torch.stack(errors).view(-1, 2)
    m = beta * (ratios[:, 0] - ratios[:, 1])
    em = beta * errors.sum(1) + 2 ** -22 * m.abs()
    f = torch.nn.functional.logsigmoid
    loss = -(1 - smooth) * f(m) - smooth * f(-m)
    sigma = torch.sigmoid(-m)
    w = torch.zeros_like(head.logp)
    dw = torch.zeros_like(head.logp)
    for p in range(m.shape[0]):
        for s, sign in ((0, 1.0), (1, -1.0)):
            rows = slice(at[2 * p + s], at[2 * p + s + 1])
            w[rows] = sign * beta * (sigma[p] - smooth) / counts[2 * p + s]
            dw[rows] = beta * (em[p] / 4 + 2 ** -20) / counts[2 * p + s]
    return (loss, em + 2 ** -20 * (loss.abs() + 1), ratios, errors + 2 ** -23 * ratios.abs(), w, dw)


def batch(T, V, D, pairs, layout, seed, pad=0, offset=0, tail=0):
    x, w = operands(T, V, D, layout, seed, pad=pad, offset=offset)
    target = targets(T, V, seed + 1)
    g = gen(seed + 2)
    cuts = (torch.rand(2 * pairs + 1, generator=g, device="cuda") * (T - tail + 1)).long().sort().values
    reference = -math.log(V) + torch.randn(T, generator=g, device="cuda")
    return x, w, target, cuts.clamp_max(T - tail), reference


SIZES = [(1, 2, 8, 1), (2, 7, 3, 1), (5, 1000, 64, 2), (7, 100, 17, 4), (64, 4099, 96, 3),
         (66, 300, 520, 33), (130, 255, 257, 5), (300, 2048, 64, 1), (513, 777, 130, 40)]


@pytest.mark.parametrize("layout", [VOCAB, WIDTH])
@pytest.mark.parametrize("T,V,D,pairs", SIZES)
@pytest.mark.parametrize("beta,smooth,average,with_reference,scale", [
    (0.1, 0.0, False, True, 1.0), (0.5, 0.2, True, True, 0.7), (2.0, 0.1, False, False, 1.0)])
def test_preference(T, V, D, pairs, beta, smooth, average, with_reference, scale, layout):
    x, w, target, offsets, reference = batch(T, V, D, pairs, layout, 30, tail=min(2, T // 8))
    reference = reference if with_reference else None
    args = dict(reference=reference, beta=beta, label_smoothing=smooth, average=average,
                logit_scale=scale, layout=layout)
    head = Head(x, w, target, layout, scale)
    loss, el, ratios, er, slope, es = pair_reference(head, target, offsets, reference, beta, smooth, average)
    dloss = torch.rand(pairs, generator=gen(33), device="cuda") + 0.5
    per_row = torch.zeros_like(slope)
    at = offsets.tolist()
    for p in range(pairs):
        per_row[at[2 * p]:at[2 * p + 2]] = dloss[p].to(D64)
    only = tg.linear_preference(x, w, target, offsets, **args)
    step = tg.linear_preference_step(x, w, target, offsets, dloss, **args)
    pieces = tg.linear_preference_step(x, w, target, offsets, dloss, piece_rows=max(1, T // 3), **args)
    for got in (only, step, pieces):
        assert got[0].shape == (pairs,) and got[1].shape == (pairs, 2)
        assert ((got[0].to(D64) - loss).abs() <= el).all()
        assert ((got[1].to(D64) - ratios).abs() <= er).all()
    for got in (step, pieces):
        head.check_grads(slope * per_row, es * per_row, *got[2:])
        outside = torch.ones(T, dtype=torch.bool, device="cuda")
        outside[at[0]:at[-1]] = False
        assert (got[2][outside | ~head.live] == 0).all()


def policy_inputs(head, T, seed, low, high, advantages=True):
    g = gen(seed)
    moved = 0.3 * torch.randn(T, generator=g, device="cuda", dtype=D64)
    for border in (math.log(1 - low) if low < 1 else -9.0, math.log(1 + high)):
        near = (moved - border).abs() < 0.02
        moved = torch.where(near, moved + 0.05, moved)
    old = (head.logp - moved).float()
    advantage = torch.randn(T, generator=g, device="cuda")
    advantage[::7] = 0.0
    reference = (head.logp + 0.3 * torch.randn(T, generator=g, device="cuda", dtype=D64)).float()
    return old, advantage, reference


def policy_reference(head, old, advantage, reference, low, high, kl):
    """(loss, its error, weight of each row for dloss 1, its error)"""
    a = advantage.to(D64)
    r = torch.exp(head.logp - old.to(D64))
    er = r * (head.e + 2 ** -20 * (1 + (head.logp - old).abs()))
    first, second = r * a, r.clamp(1 - low, 1 + high) * a
    loss, el = -torch.minimum(first, second), er * a.abs()
    active = first <= second
    w = torch.where(active, r * a, torch.zeros_like(a))
    ew = torch.where(active, er * a.abs(), torch.zeros_like(a))
    if kl:
        d = reference.to(D64) - head.logp
        ed = head.e + 2 ** -22 * d.abs()
        loss = loss + kl * (torch.expm1(d) - d)
        el = el + kl * (torch.expm1(d).abs() * ed + 2 ** -20 * (torch.exp(d) + d.abs() + 1))
        w = w + kl * torch.expm1(d)
        ew = ew + kl * torch.exp(d) * (ed + 2 ** -20)
    zero = torch.zeros_like(loss)
    return (torch.where(head.live, loss, zero), el + 2 ** -22 * (loss.abs() + 1), w,
            ew + 2 ** -22 * w.abs())


@pytest.mark.parametrize("layout", [VOCAB, WIDTH])
@pytest.mark.parametrize("T,V,D", [s[:3] for s in SIZES])
@pytest.mark.parametrize("low,high,kl,scale", [(0.2, 0.2, 0.0, 1.0), (0.1, 0.4, 0.2, 0.7), (1.0, 0.0, 0.05, 1.3)])
def test_policy(T, V, D, low, high, kl, scale, layout):
    x, w = operands(T, V, D, layout, 40)
    target = targets(T, V, 41)
    head = Head(x, w, target, layout, scale)
    old, advantage, reference = policy_inputs(head, T, 42, low, high)
    loss, el, weight, ew = policy_reference(head, old, advantage, reference, low, high, kl)
    dloss = torch.rand(T, generator=gen(43), device="cuda") + 0.5
    args = dict(reference=reference if kl else None, clip_low=low, clip_high=high, kl_weight=kl,
                logit_scale=scale, layout=layout)
    only = tg.linear_policy(x, w, target, old, advantage, **args)
    step = tg.linear_policy_step(x, w, target, old, advantage, dloss, **args)
    pieces = tg.linear_policy_step(x, w, target, old, advantage, dloss, piece_rows=max(1, T // 3), **args)
    for got in (only, step, pieces):
        assert ((got[0].to(D64) - loss).abs() <= el).all()
        assert ((got[1].to(D64) - head.logp).abs() <= head.e).all()
        assert (got[0][~head.live] == 0).all() and (got[1][~head.live] == 0).all()
    for got in (step, pieces):
        head.check_grads(weight * dloss.to(D64), ew * dloss.to(D64), *got[2:])


@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 8), (1, 0)])
@pytest.mark.parametrize("layout", [VOCAB, WIDTH])
def test_strides(pad, offset, layout):
    T, V, D, pairs = 90, 700, 77, 6
    x, w, target, offsets, reference = batch(T, V, D, pairs, layout, 50, pad, offset)
    head = Head(x, w, target, layout)
    loss, el, _, _, slope, es = pair_reference(head, target, offsets, reference, 0.3, 0.0, False)
    got = tg.linear_preference_step(x, w, target, offsets, torch.ones(pairs, device="cuda"),
                                    reference=reference, beta=0.3, layout=layout)
    assert ((got[0].to(D64) - loss).abs() <= el).all()
    head.check_grads(slope, es, *got[2:])


@pytest.mark.parametrize("layout", [VOCAB, WIDTH])
@pytest.mark.parametrize("T,V,D,pad,offset", [
    (600, 3001, 1001, 0, 0), (300, 5003, 777, 3, 1), (3, 9001, 601, 0, 0), (1500, 2501, 259, 1, 3),
    (130, 20001, 65, 0, 0)])
def test_rows_that_start_anywhere(T, V, D, pad, offset, layout):
    """Gradients whose rows TMA cannot store, from few tokens to tiles of a pair, whole and summed over pieces."""
    x, w, target, offsets, reference = batch(T, V, D, 1, layout, 150, pad, offset)
    head = Head(x, w, target, layout)
    advantage, old = torch.randn(T, generator=gen(151), device="cuda"), head.logp.float()
    loss, el, weight, ew = policy_reference(head, old, advantage, reference, 0.2, 0.2, 0.0)
    for piece_rows in (0, T // 2 + 1):
        got = tg.linear_policy_step(x, w, target, old, advantage, torch.ones(T, device="cuda"), layout=layout,
                                    piece_rows=piece_rows)
        assert ((got[0].to(D64) - loss).abs() <= el).all()
        head.check_grads(weight, ew, *got[2:])


@pytest.mark.parametrize("piece_rows", [0, 16])
def test_empty_and_ignored(piece_rows):
    """Empty sequences, sequences of ignored rows alone, no pairs at all, no rows at all."""
    T, V, D = 40, 300, 64
    x, w, target, _, reference = batch(T, V, D, 1, VOCAB, 60)
    target[10:20] = IGNORE
    offsets = torch.tensor([0, 0, 0, 5, 5, 10, 20, 20, 40], device="cuda")
    head = Head(x, w, target, VOCAB)
    for average in (False, True):
        loss, el, ratios, er, slope, es = pair_reference(head, target, offsets, reference, 0.1, 0.0, average)
        got = tg.linear_preference_step(x, w, target, offsets, torch.ones(4, device="cuda"), average=average,
                                        reference=reference, piece_rows=piece_rows)
        assert ((got[0].to(D64) - loss).abs() <= el).all() and abs(float(got[0][0]) - math.log(2)) < 1e-6
        assert ((got[1].to(D64) - ratios).abs() <= er).all() and (got[1][0] == 0).all()
        head.check_grads(slope, es, *got[2:])
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    loss, ratios, dx, dw = tg.linear_preference_step(x, w, target, none, torch.ones(0, device="cuda"),
                                                     piece_rows=piece_rows)
    assert loss.shape == (0,) and ratios.shape == (0, 2) and (dx == 0).all() and (dw == 0).all()
    zeros = torch.zeros(3, dtype=torch.int64, device="cuda")
    loss, ratios, dx, dw = tg.linear_preference_step(x[:0], w, target[:0], zeros, torch.ones(1, device="cuda"),
                                                     piece_rows=piece_rows)
    assert abs(float(loss[0]) - math.log(2)) < 1e-6 and dx.shape == (0, D) and (dw == 0).all()
    empty = torch.zeros(0, device="cuda")
    loss, logp, dx, dw = tg.linear_policy_step(x[:0], w, target[:0], empty, empty, empty,
                                               piece_rows=piece_rows)
    assert loss.shape == logp.shape == (0,) and dx.shape == (0, D) and (dw == 0).all()
    target[:] = IGNORE
    v = torch.ones(T, device="cuda")
    loss, logp, dx, dw = tg.linear_policy_step(x, w, target, v, v, v, piece_rows=piece_rows)
    assert all((t == 0).all() for t in (loss, logp, dx, dw))


@pytest.mark.parametrize("piece_rows", [0, 16])
@pytest.mark.parametrize("bad", [[0, 30, 20, 35, 40], [-3, 10, 20, 30, 40], [0, 10, 20, 30, 41],
                                 [0, 10, 20, 30, 2 ** 62], [0, -2 ** 62, 20, 30, 40]])
def test_bad_offsets(bad, piece_rows):
    """Offsets that decrease or leave the rows: those pairs and the gradients are NaN, other pairs' losses
    are not, and nothing else happens."""
    T, V, D = 40, 300, 64
    x, w, target, _, reference = batch(T, V, D, 1, VOCAB, 70)
    offsets = torch.tensor(bad, device="cuda")
    good = [0 <= bad[2 * p] <= bad[2 * p + 1] <= bad[2 * p + 2] <= T for p in range(2)]
    loss, ratios, dx, dw = tg.linear_preference_step(x, w, target, offsets, torch.ones(2, device="cuda"),
                                                     reference=reference, piece_rows=piece_rows)
    live = target != IGNORE
    assert loss.isnan().tolist() == [not g for g in good] == ratios.isnan().all(1).tolist()
    assert dx[live].isnan().all() and (dx[~live] == 0).all() and dw.isnan().all()


@pytest.mark.parametrize("piece_rows", [0, 16])
def test_bad_targets_and_values(piece_rows):
    """A target outside of the vocabulary, and values that are not finite, show as NaN in their rows (or
    pairs) and in the sums over rows."""
    T, V, D = 40, 300, 64
    x, w, target, _, reference = batch(T, V, D, 1, VOCAB, 80)
    offsets = torch.tensor([0, 10, 20, 30, 36], device="cuda")
    target[:] = 5
    target[3] = V
    ones = torch.ones(2, device="cuda")
    loss, ratios, dx, dw = tg.linear_preference_step(x, w, target, offsets, ones, reference=reference,
                                                     piece_rows=piece_rows)
    assert loss.isnan().tolist() == [True, False] and ratios.isnan().tolist() == [[True, False], [False, False]]
    assert dx[:20].isnan().all() and dx[20:].isfinite().all() and dw.isnan().any()
    target[3] = 5
    reference[25] = math.nan
    loss, _, dx, _ = tg.linear_preference_step(x, w, target, offsets, ones, reference=reference,
                                               piece_rows=piece_rows)
    assert loss.isnan().tolist() == [False, True]
    assert dx[20:36].isnan().all() and dx[:20].isfinite().all() and (dx[36:] == 0).all()
    v = torch.ones(T, device="cuda")
    old = torch.full((T,), -5.0, device="cuda")
    advantage = v.clone()
    old[4], advantage[9] = math.nan, math.nan
    old[12], advantage[12] = -1e4, 1.0     # an infinite ratio: clipped
    target[20] = -7
    loss, logp, dx, dw = tg.linear_policy_step(x, w, target, old, advantage, v, piece_rows=piece_rows)
    rows = torch.zeros(T, dtype=torch.bool, device="cuda")
    rows[[4, 9, 20]] = True
    assert torch.equal(loss.isnan(), rows) and torch.equal(dx.isnan().all(1), rows)
    assert abs(float(loss[12]) + 1.2) < 1e-6 and (dx[12] == 0).all() and dw.isnan().any()


@pytest.mark.parametrize("piece_rows", [0, 16])
def test_infinite_references(piece_rows):
    """A reference that held a token impossible: the margin is infinite, and the losses and gradients are
    their limits."""
    T, V, D = 40, 300, 64
    x, w, target, _, reference = batch(T, V, D, 1, VOCAB, 160)
    target[:] = 7
    offsets = torch.tensor([0, 10, 20, 30, 40], device="cuda")
    reference[3] = -math.inf   # the chosen of pair 0: infinitely ahead
    reference[25] = -math.inf  # the chosen of pair 1
    reference[35] = -math.inf  # and its rejected: no order between them
    loss, ratios, dx, _ = tg.linear_preference_step(x, w, target, offsets, torch.ones(2, device="cuda"),
                                                    reference=reference, piece_rows=piece_rows)
    assert float(loss[0]) == 0 and float(ratios[0, 0]) == math.inf and loss[1].isnan()
    assert (dx[:20] == 0).all() and dx[20:].isnan().all()
    loss, _, dx, _ = tg.linear_preference_step(x[:20], w, target[:20], offsets[[0, 0, 1, 1, 2]].contiguous(),
                                               torch.ones(2, device="cuda"), reference=reference[:20].contiguous(),
                                               piece_rows=piece_rows)
    assert loss[0] == math.inf and loss[1].isfinite() and dx.isfinite().all()
    one = torch.ones(T, device="cuda")
    reference[5] = math.inf
    loss, logp, _, _ = tg.linear_policy_step(x, w, target, one, one, one, reference=reference, kl_weight=0.1,
                                             piece_rows=piece_rows)
    assert loss[5] == math.inf and loss[3] == math.inf and loss[[0, 1, 2, 4]].isfinite().all()


@pytest.mark.parametrize("V,D", [(1710, 80), (7033, 360), (30666, 768), (7033, 1596)])
def test_log_probabilities_lean_neither_way(V, D):
    """The mean error over many tokens, which a sum over a sequence multiplies: 5e-8 and three standard errors of 4096
    tokens whose errors are 1.3e-6 (2^-24 of up to 8 for each of a logit's few roundings), 1.1e-7 in all."""
    T = 4096
    g = gen(170)
    x = torch.randn(T, D, generator=g, device="cuda").half()
    w = (torch.randn(V, D, generator=g, device="cuda") * (2 / math.sqrt(D))).half()
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    one = torch.zeros(T, device="cuda")
    _, logp = tg.linear_policy(x, w, target, one, one)
    error = torch.empty(T, dtype=D64, device="cuda")
    for a in range(0, T, 1024):
        z = x[a:a + 1024].to(D64) @ w.to(D64).t()
        error[a:a + 1024] = logp[a:a + 1024] - torch.log_softmax(z, 1).gather(1, target[a:a + 1024, None])[:, 0]
    assert abs(float(error.mean())) < 1.1e-7 and float(error.square().mean().sqrt()) < 1.6e-6


def test_long_answers():
    """Sums of long answers that nearly cancel keep their difference; an answer that is far behind or
    ahead."""
    T, V, D = 6000, 64, 16
    x, w = operands(T, V, D, VOCAB, 90)
    target = targets(T, V, 91, 0.0)
    head = Head(x, w, target, VOCAB)
    offsets = torch.tensor([0, 3000, 6000], device="cuda")
    for shift in (0.0, 0.5, -0.5):
        reference = (head.logp - 0.001).float()
        reference[:3000] -= shift
        for beta in (0.1, 1.0):
            loss, el, ratios, er, slope, es = pair_reference(head, target, offsets, reference, beta, 0.0, False)
            got = tg.linear_preference_step(x, w, target, offsets, torch.full((1,), 64.0, device="cuda"),
                                            reference=reference, beta=beta)
            assert ((got[0].to(D64) - loss).abs() <= el).all() and ((got[1].to(D64) - ratios).abs() <= er).all()
            head.check_grads(64 * slope, 64 * es, *got[2:])


def test_many_pairs():
    """More pairs than rows of a block, of a row each, over several pieces of a kind."""
    T, V, D, pairs = 3000, 96, 24, 1500
    x, w = operands(T, V, D, VOCAB, 95)
    target = targets(T, V, 96, 0.1)
    offsets = torch.arange(2 * pairs + 1, device="cuda")
    head = Head(x, w, target, VOCAB)
    loss, el, _, _, slope, es = pair_reference(head, target, offsets, None, 0.7, 0.0, False)
    for piece_rows in (0, 700):
        got = tg.linear_preference_step(x, w, target, offsets, torch.ones(pairs, device="cuda"), beta=0.7,
                                        piece_rows=piece_rows)
        assert ((got[0].to(D64) - loss).abs() <= el).all()
        head.check_grads(slope, es, *got[2:])


@pytest.mark.parametrize("T,V,D", [(64, 28672, 512), (200, 1000, 96), (16, 20000, 1024)])
def test_same_bits_again_captured_and_on_a_stream(T, V, D):
    x, w, target, offsets, reference = batch(T, V, D, 3, VOCAB, 100)
    old, advantage = reference + 0.1, torch.randn(T, generator=gen(101), device="cuda")
    dloss, dpair = torch.ones(T, device="cuda"), torch.ones(3, device="cuda")

    def step(stream=None):
        return (*tg.linear_preference_step(x, w, target, offsets, dpair, reference=reference, stream=stream),
                *tg.linear_policy_step(x, w, target, old, advantage, dloss, reference=reference,
                                       kl_weight=0.1, stream=stream),
                *tg.linear_preference(x, w, target, offsets, reference=reference, stream=stream),
                *tg.linear_preference_step(x, w, target, offsets, dpair, piece_rows=T // 2, stream=stream))

    want = step()
    for a, b in zip(want, step()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
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


def test_against_cross_entropy():
    """A policy step whose ratios are 1 has cross entropy's gradients with the advantages as weights."""
    T, V, D = 150, 900, 128
    x, w = operands(T, V, D, VOCAB, 110)
    target = targets(T, V, 111)
    live = target != IGNORE
    weights = torch.rand(T, generator=gen(112), device="cuda") + 0.1
    one = torch.ones(T, device="cuda")
    _, logp = tg.linear_policy(x, w, target, one, weights)
    nll = tg.linear_cross_entropy(x, w, target)
    head = Head(x, w, target, VOCAB)
    assert ((logp + nll).to(D64).abs() <= 2 * head.e).all()
    loss, again, dx, dw = tg.linear_policy_step(x, w, target, logp, weights, one)
    assert torch.equal(logp, again)
    assert torch.equal(loss, torch.where(live, -weights, torch.zeros_like(loss)))
    zero = torch.zeros(T, dtype=D64, device="cuda")
    head.check_grads(weights.to(D64), zero, dx, dw)
    head.check_grads(weights.to(D64), zero, *tg.linear_cross_entropy_step(x, w, target, weights)[1:])


def test_autograd():
    T, V, D, pairs = 60, 500, 64, 3
    x, w, target, offsets, reference = batch(T, V, D, pairs, VOCAB, 120)
    xg, wg = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss, ratios = autograd.linear_preference(xg, wg, target, offsets, reference, beta=0.2, label_smoothing=0.1)
    assert not ratios.requires_grad
    (loss * 512).backward()
    want = tg.linear_preference_step(x, w, target, offsets, torch.full((pairs,), 512 / pairs, device="cuda"),
                                     reference=reference, beta=0.2, label_smoothing=0.1)
    assert torch.allclose(loss, want[0].mean(), atol=1e-6)
    for a, b in ((xg.grad, want[2]), (wg.grad, want[3])):
        # 512 / 3 is rounded on either way
        assert ((a.float() - b.float()).abs() <= 2 ** -10 * b.float().abs() + 2 ** -12 * b.float().abs().max()).all()
    old, advantage = reference, torch.randn(T, generator=gen(121), device="cuda")
    xg.grad = wg.grad = None
    loss, logp = autograd.linear_policy(xg, wg, target, old, advantage, reference, kl_weight=0.1,
                                        reduction="sum")
    loss.backward()
    want = tg.linear_policy_step(x, w, target, old, advantage, torch.ones(T, device="cuda"),
                                 reference=reference, kl_weight=0.1)
    assert torch.equal(xg.grad, want[2]) and torch.equal(wg.grad, want[3]) and torch.equal(logp, want[1])
    with pytest.raises(ValueError, match="detach"):
        autograd.linear_policy(xg, wg, target, old.clone().requires_grad_(True), advantage)
    with pytest.raises(ValueError, match="detach"):
        autograd.linear_preference(xg, wg, target, offsets, reference.clone().requires_grad_(True))
    loss, _ = autograd.linear_policy(xg, wg, target, old, advantage)
    only, = torch.autograd.grad(loss, xg, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated again"):
        only.float().sum().backward()


def test_differences():
    """The gradients against differences of the loss by its formula in 64 bits."""
    T, V, D, pairs = 24, 50, 32, 3
    x, w, target, offsets, reference = batch(T, V, D, pairs, VOCAB, 130)
    head = Head(x, w, target, VOCAB)
    old, advantage, other = policy_inputs(head, T, 131, 0.2, 0.2)
    pair = tg.linear_preference_step(x, w, target, offsets, torch.ones(pairs, device="cuda"),
                                     reference=reference, beta=0.5)
    policy = tg.linear_policy_step(x, w, target, old, advantage, torch.ones(T, device="cuda"),
                                   reference=other, kl_weight=0.1)

    def losses(xv, wv):
        h = Head(xv, wv, target, VOCAB)
        return (pair_reference(h, target, offsets, reference, 0.5, 0.0, False)[0].sum(),
                policy_reference(h, old, advantage, other, 0.2, 0.2, 0.1)[0].sum())

    for i in range(2):
        way = torch.randn((x, w)[i].shape, generator=gen(132 + i), device="cuda").to(D64)
        eps = 1e-6
        up = losses(*(t.to(D64) + (eps * way if j == i else 0) for j, t in enumerate((x, w))))
        down = losses(*(t.to(D64) - (eps * way if j == i else 0) for j, t in enumerate((x, w))))
        for grads, a, b in ((pair, up[0], down[0]), (policy, up[1], down[1])):
            got = grads[2 + i].to(D64) * way
            # G and the result are each rounded to fp16
            assert (got.sum() - (a - b) / (2 * eps)).abs() <= 2 ** -9 * got.abs().sum()


def test_refusals():
    T, V, D = 12, 40, 16
    x, w, target, offsets, reference = batch(T, V, D, 2, VOCAB, 140)
    v = torch.ones(T, device="cuda")
    for kw in (dict(beta=0.0), dict(beta=math.inf), dict(label_smoothing=1.0), dict(label_smoothing=-0.1)):
        with pytest.raises(tg.TgError):
            tg.linear_preference(x, w, target, offsets, **kw)
    for bad in (offsets[:-1], offsets.int(), offsets[None], offsets.cpu()):
        with pytest.raises((ValueError, TypeError)):
            tg.linear_preference(x, w, target, bad)
    with pytest.raises(ValueError):
        tg.linear_preference(x, w, target, offsets, reference[:-1])
    with pytest.raises(TypeError):
        tg.linear_preference(x, w, target, offsets, reference.half())
    with pytest.raises(ValueError):
        tg.linear_preference_step(x, w, target, offsets, v)
    for kw in (dict(clip_low=1.5), dict(clip_low=-0.1), dict(clip_high=-0.1), dict(kl_weight=-1.0, reference=v),
               dict(clip_high=math.nan), dict(logit_scale=0.0)):
        with pytest.raises(tg.TgError):
            tg.linear_policy(x, w, target, v, v, **kw)
    with pytest.raises(ValueError):
        tg.linear_policy(x, w, target, v, v, kl_weight=0.1)
    with pytest.raises(ValueError):
        tg.linear_policy(x, w, target, v[1:], v)
    with pytest.raises(TypeError):
        tg.linear_policy(x, w, target, v.double(), v)
