"""Layer norm and the head's losses at the C ABI without a GPU: what they refuse on the host, and the
layout of the options."""

import ctypes

import pytest

from fp16_gemm_relu_gb300 import binding as b

P = 4096  # a pointer that is never followed: every call here ends on the host


@pytest.fixture(scope="module", autouse=True)
def lib():
    from fp16_gemm_relu_gb300 import build

    build.build()
    return b.load_library()


def norm(**kw):
    a = dict(X=P, gamma=P, beta=P, Y=P, mean=P, rstd=P, M=4, N=16, ldx=16, ldy=16, eps=1e-5,
             param_type=b.TG_TYPE_F16)
    a.update(kw)
    return b.tg_layernorm_f16(**a)


def norm_backward(**kw):
    a = dict(dY=P, X=P, gamma=P, mean=P, rstd=P, dX=P, dgamma=P, dbeta=P, M=4, N=16, lddy=16,
             ldx=16, lddx=16, param_type=b.TG_TYPE_F16)
    a.update(kw)
    return b.tg_layernorm_backward_f16(**a)


def cross_entropy(**kw):
    a = dict(X=P, W=P, target=P, ignore_index=-100, logit_scale=1.0, dloss=P, loss=P, lse=P, dX=P,
             dW=P, T=4, V=32, D=16, ldx=16, ldw=16, lddx=16, lddw=16, options=None)
    a.update(kw)
    return b.tg_linear_cross_entropy_f16(**a)


def distill(**kw):
    a = dict(X=P, W=P, teacher_index=P, teacher_logits=P, teacher_type=b.TG_TYPE_F16, top=8, ldt=8,
             temperature=1.0, dloss=P, loss=P, lse=P, dX=P, dW=P, T=4, V=32, D=16, ldx=16, ldw=16,
             lddx=16, lddw=16, options=None)
    a.update(kw)
    return b.tg_linear_distill_f16(**a)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(N=32769, ldx=32769, ldy=32769), dict(ldx=15), dict(ldy=15),
    dict(eps=-1.0), dict(eps=float("nan")), dict(param_type=2), dict(X=0), dict(Y=0)])
def test_norm_refuses(bad):
    assert norm(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(N=32769, lddy=32769, ldx=32769, lddx=32769), dict(lddy=15),
    dict(ldx=15), dict(lddx=15), dict(param_type=-1), dict(X=0), dict(dY=0), dict(mean=0),
    dict(rstd=0)])
def test_norm_backward_refuses(bad):
    assert norm_backward(**bad) == b.TG_ERR_INVALID_ARG


def test_norm_misaligned():
    for k in ("X", "Y", "gamma", "beta"):
        assert norm(**{k: P + 1}) == b.TG_ERR_MISALIGNED
    for k in ("mean", "rstd"):
        assert norm(**{k: P + 2}) == b.TG_ERR_MISALIGNED
    assert norm(gamma=P + 2, param_type=b.TG_TYPE_F32) == b.TG_ERR_MISALIGNED
    for k in ("X", "dY", "dX", "gamma", "dgamma", "dbeta"):
        assert norm_backward(**{k: P + 1}) == b.TG_ERR_MISALIGNED
    assert norm_backward(dbeta=P + 2, param_type=b.TG_TYPE_F32) == b.TG_ERR_MISALIGNED


def test_norm_nothing_to_do():
    assert norm(M=0, X=0, Y=0) == b.TG_OK
    assert norm_backward(dX=0, dgamma=0, dbeta=0) == b.TG_OK


BAD_HEAD = [
    dict(T=-1), dict(V=0), dict(D=0), dict(T=2 ** 31), dict(V=2 ** 31), dict(ldx=15),
    dict(T=2 ** 30, V=2 ** 30, D=2 ** 30, ldx=2 ** 30, ldw=2 ** 30, lddx=2 ** 30, lddw=2 ** 30),
    dict(ldw=15), dict(lddx=15), dict(lddw=15), dict(X=0), dict(W=0), dict(dloss=0),
    dict(options={"layout": 2}), dict(options={"layout": 1}),  # width-major: ldw >= V
    dict(options={"piece_rows": -1}), dict(options={"timeout_ms": -1})]


@pytest.mark.parametrize("bad", BAD_HEAD + [
    dict(target=0), dict(logit_scale=0.0), dict(logit_scale=-1.0), dict(logit_scale=float("nan")),
    dict(logit_scale=float("inf"))])
def test_cross_entropy_refuses(bad):
    assert cross_entropy(**bad) == b.TG_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", BAD_HEAD + [
    dict(teacher_index=0), dict(teacher_logits=0), dict(top=0), dict(top=1025, ldt=1025),
    dict(ldt=7), dict(temperature=0.0), dict(temperature=-2.0), dict(temperature=float("nan")),
    dict(temperature=float("inf")), dict(temperature=1e-40), dict(teacher_type=5)])
def test_distill_refuses(bad):
    assert distill(**bad) == b.TG_ERR_INVALID_ARG


def test_head_misaligned():
    for k in ("X", "W", "dX", "dW"):
        assert cross_entropy(**{k: P + 1}) == b.TG_ERR_MISALIGNED
        assert distill(**{k: P + 1}) == b.TG_ERR_MISALIGNED
    for k in ("loss", "lse", "dloss"):
        assert cross_entropy(**{k: P + 2}) == b.TG_ERR_MISALIGNED
    assert cross_entropy(target=P + 4) == b.TG_ERR_MISALIGNED
    assert distill(teacher_index=P + 4) == b.TG_ERR_MISALIGNED
    assert distill(teacher_logits=P + 1) == b.TG_ERR_MISALIGNED
    assert distill(teacher_logits=P + 2, teacher_type=b.TG_TYPE_F32) == b.TG_ERR_MISALIGNED


def test_head_no_rows_without_weight_gradient():
    assert cross_entropy(T=0, X=0, target=0, dloss=0, dW=0) == b.TG_OK
    assert distill(T=0, X=0, teacher_index=0, teacher_logits=0, dloss=0, dW=0) == b.TG_OK


def test_options_layout():
    assert ctypes.sizeof(b.tg_head_options) == 24
    with pytest.raises(KeyError):
        cross_entropy(options={"no_such_option": 1})
