"""The gated product, the preference and policy losses and the clipping of gradients at the C ABI without a
GPU: what they refuse on the host."""

import ctypes
import math

import pytest

from fp16_gemm_relu_gb300 import binding as b

P = 4096  # a pointer that is never followed: every call here ends on the host
FAR = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    from fp16_gemm_relu_gb300 import build

    build.build()
    return b.load_library()


def gated(**kw):
    a = dict(X=P, Wg=P, Wu=P, H=P, gate=P, up=P, activation=b.TG_ACT_SILU, trans_w=0, M=4, N=16, K=24,
             ldx=24, ldwg=24, ldwu=24, ldh=16, ldgate=16, ldup=16)
    a.update(kw)
    return b.tg_gated_f16(**a)


def gated_backward(**kw):
    a = dict(dH=P, X=P, Wg=P, Wu=P, gate=P, up=P, dX=P, dWg=P, dWu=P, activation=b.TG_ACT_SILU,
             trans_w=0, M=4, N=16, K=24, lddh=16, ldx=24, ldwg=24, ldwu=24, ldgate=16, ldup=16, lddx=24,
             lddwg=24, lddwu=24)
    a.update(kw)
    return b.tg_gated_backward_f16(**a)


def preference(**kw):
    a = dict(X=P, W=P, target=P, ignore_index=-100, logit_scale=1.0, offsets=P, pairs=2, reference=P,
             beta=0.1, label_smoothing=0.0, average=0, dloss=P, loss=P, ratios=P, dX=P, dW=P, T=4, V=32,
             D=16, ldx=16, ldw=16, lddx=16, lddw=16)
    a.update(kw)
    return b.tg_linear_preference_f16(**a)


def policy(**kw):
    a = dict(X=P, W=P, target=P, ignore_index=-100, logit_scale=1.0, old_logp=P, advantage=P,
             reference=P, clip_low=0.2, clip_high=0.2, kl_weight=0.1, dloss=P, loss=P, logp=P, dX=P, dW=P,
             T=4, V=32, D=16, ldx=16, ldw=16, lddx=16, lddw=16)
    a.update(kw)
    return b.tg_linear_policy_f16(**a)


def clip(*grads, loss_scale=1.0, max_norm=1.0, norm=P):
    return b.tg_clip_gradients([b.tg_gradient(*g) for g in grads], loss_scale, max_norm, norm)


BIG = (1 << 29) + 1
HALF = 1 << 28


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(M=BIG), dict(N=BIG, ldwg=BIG, ldwu=BIG, ldh=BIG, ldgate=BIG,
                                                        ldup=BIG),
    dict(ldx=23), dict(ldwg=15), dict(ldwu=15), dict(trans_w=1, ldwg=23), dict(trans_w=2), dict(ldh=15),
    dict(ldgate=15), dict(ldup=15), dict(activation=5), dict(activation=-1), dict(X=0), dict(Wg=0),
    dict(Wu=0), dict(H=0), dict(ldx=1 << 37),
    dict(M=HALF, N=HALF, ldwg=HALF, ldwu=HALF, ldh=HALF, ldgate=HALF, ldup=HALF)])
def test_gated_refuses(bad):
    assert gated(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", ["X", "Wg", "Wu", "H", "gate", "up"])
def test_gated_misaligned(bad):
    assert gated(**{bad: P + 1}) == b.TG_ERR_MISALIGNED


def test_gated_nothing_to_do():
    assert gated(M=0, X=0, Wg=0, Wu=0, H=0) == b.TG_OK
    assert gated_backward(dX=0, dWg=0, dWu=0) == b.TG_OK


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(ldx=23), dict(ldwg=15), dict(lddh=15), dict(ldgate=15),
    dict(ldup=15), dict(lddx=23), dict(lddwg=15), dict(lddwu=15), dict(activation=5), dict(dH=0),
    dict(X=0), dict(gate=0), dict(up=0), dict(Wg=0), dict(trans_w=-1)])
def test_gated_backward_refuses(bad):
    assert gated_backward(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", ["dH", "X", "Wg", "Wu", "gate", "up", "dX", "dWg", "dWu"])
def test_gated_backward_misaligned(bad):
    assert gated_backward(**{bad: P + 1}) == b.TG_ERR_MISALIGNED


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(V=0), dict(D=0), dict(ldx=15), dict(ldw=15), dict(pairs=-1), dict(pairs=1 << 31),
    dict(offsets=0), dict(beta=0.0), dict(beta=-1.0), dict(beta=math.nan), dict(beta=math.inf),
    dict(label_smoothing=1.0), dict(label_smoothing=-0.5), dict(label_smoothing=math.nan), dict(dloss=0),
    dict(X=0), dict(target=0), dict(logit_scale=0.0), dict(lddx=15), dict(lddw=15)])
def test_preference_refuses(bad):
    assert preference(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(offsets=P + 4), dict(reference=P + 2), dict(dloss=P + 1),
                                 dict(loss=P + 2), dict(ratios=P + 2), dict(target=P + 4), dict(X=P + 1)])
def test_preference_misaligned(bad):
    assert preference(**bad) == b.TG_ERR_MISALIGNED


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(V=0), dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_high=-0.1),
    dict(clip_low=math.nan), dict(clip_high=math.inf), dict(kl_weight=-0.1), dict(kl_weight=math.nan),
    dict(reference=0), dict(old_logp=0), dict(advantage=0), dict(dloss=0), dict(target=0)])
def test_policy_refuses(bad):
    assert policy(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(old_logp=P + 2), dict(advantage=P + 1), dict(reference=P + 2),
                                 dict(loss=P + 2), dict(logp=P + 2)])
def test_policy_misaligned(bad):
    assert policy(**bad) == b.TG_ERR_MISALIGNED


@pytest.mark.parametrize("grads", [
    [(P, FAR, -1, 0, 0)], [(0, FAR, 4, 0, 0)], [(P, FAR, 4, 2, 0)], [(P, FAR, 4, 0, 3)],
    [(P, FAR, 4, 0, 0), (P + 64, 0, 4, 0, 0)],                  # an output here and none there
    [(P, FAR, 4, 0, 0), (P + 64, FAR + 6, 4, 0, 0)],            # outputs that overlap
    [(P, FAR, 4, 0, 0), (P + 64, P, 4, 0, 0)],                  # an output over another gradient
    [(P, P, 4, 0, 1)], [(P, P + 4, 4, 0, 0)], [(P, P - 4, 4, 0, 0)],
    [(P, P, 4, 0, 0), (P, P, 4, 0, 0)]])
def test_clip_refuses(grads):
    assert clip(*grads) == b.TG_ERR_INVALID_ARG


def test_clip_arguments():
    g = (P, FAR, 4, 0, 0)
    assert clip(g, norm=0) == b.TG_ERR_INVALID_ARG
    assert clip(g, loss_scale=0.0) == b.TG_ERR_INVALID_ARG
    assert clip(g, loss_scale=math.inf) == b.TG_ERR_INVALID_ARG
    assert clip(g, max_norm=-1.0) == b.TG_ERR_INVALID_ARG
    assert clip(g, max_norm=math.nan) == b.TG_ERR_INVALID_ARG
    assert clip(g, norm=P + 1) == b.TG_ERR_MISALIGNED
    assert clip((P + 1, FAR, 4, 0, 0)) == b.TG_ERR_MISALIGNED
    assert clip((P, FAR + 2, 4, 0, 1)) == b.TG_ERR_MISALIGNED
    assert b.load_library().tg_clip_gradients(None, 3, 1.0, 1.0, P, None) == b.TG_ERR_INVALID_ARG
    assert b.load_library().tg_clip_gradients(None, -1, 1.0, 1.0, P, None) == b.TG_ERR_INVALID_ARG


def test_layout_of_a_gradient():
    assert ctypes.sizeof(b.tg_gradient) == 32
    assert b.tg_gradient.type.offset == 24 and b.tg_gradient.out_type.offset == 28
