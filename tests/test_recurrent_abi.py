"""Host-side argument checks of the recurrent stage's C entry points: each wrong argument gives its status and a message, before
anything touches a GPU (the pointers here are never followed)."""
import ctypes

import pytest

import fourier_domain_linear_amd as eq

from test_stage_abi import BF16, INVALID, UNSUPPORTED, _at, _refused, lib  # noqa: F401


def _norm(lib, x=_at(0), residual=_at(1), gamma=_at(2), beta=_at(6), s=_at(3), y=_at(4), mean=_at(7), rstd=_at(5), N=8, C=16, G=4,  # noqa: F811
          eps=1e-6, dtype=BF16):
    return lib.eqlin_layernorm(x, residual, gamma, beta, s, y, mean, rstd, N, C, G, eps, dtype, None)


@pytest.mark.parametrize("change, want", [
    (dict(N=-1), INVALID), (dict(C=0), INVALID), (dict(G=3), INVALID), (dict(dtype=7), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x=_at(0) + 2), INVALID), (dict(y=_at(0)), INVALID), (dict(s=_at(4) + 16), INVALID), (dict(rstd=_at(5) + 1), INVALID),
    (dict(mean=_at(7) + 2), INVALID), (dict(mean=_at(5)), INVALID), (dict(beta=_at(6) + 1), INVALID), (dict(rstd=_at(1)), INVALID),
    (dict(mean=_at(4) + 64), INVALID), (dict(y=_at(6) - 16), INVALID), (dict(C=1 << 20), UNSUPPORTED), (dict(N=1 << 60), INVALID)])
def test_layernorm_refusals(lib, change, want):  # noqa: F811
    _refused(lib, _norm(lib, **change), want)


def _back(lib, s=_at(0), gamma=_at(1), mean=_at(2), rstd=_at(3), dy=_at(4), ds=_at(5), dx=_at(6), dgamma=_at(7), dbeta=_at(8), N=8, C=16,  # noqa: F811
          G=4, dtype=BF16, ws=_at(9), size=1 << 30):
    return lib.eqlin_layernorm_backward(s, gamma, mean, rstd, dy, ds, dx, dgamma, dbeta, N, C, G, dtype, ws, size, None)


@pytest.mark.parametrize("change, want", [
    (dict(N=-1), INVALID), (dict(dtype=7), INVALID), (dict(s=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), INVALID), (dict(size=4), INVALID), (dict(ws=_at(9) + 16), INVALID),
    (dict(dx=_at(0)), INVALID), (dict(dx=_at(5)), INVALID), (dict(dgamma=_at(8)), INVALID), (dict(dgamma=_at(2)), INVALID),
    (dict(dbeta=_at(6) + 32), INVALID), (dict(ws=_at(4)), INVALID), (dict(dgamma=_at(7) + 2), INVALID), (dict(dbeta=_at(8) + 1), INVALID),
    (dict(ws=None, dgamma=None), INVALID), (dict(dy=_at(4) + 8), INVALID), (dict(C=1 << 20), UNSUPPORTED),
    (dict(N=0, dgamma=_at(8)), INVALID)])
def test_layernorm_backward_refusals(lib, change, want):  # noqa: F811
    _refused(lib, _back(lib, **change), want)


def test_layernorm_of_nothing(lib):  # noqa: F811
    assert _norm(lib, N=0, x=None, y=None) == 0
    assert _back(lib, N=0, dgamma=None, dbeta=None, s=None, ws=None, size=0) == 0
    assert lib.eqlin_layernorm_backward_workspace(0, 16, 4) == 0


def _rec(**change):
    T, C, G = 100, 16, 4
    a = dict(x=_at(0), forget=_at(1), gate=_at(2), y=_at(3), state=_at(4), final=_at(5), marks=_at(6), x_token_stride=64, forget_token_stride=64,
             gate_token_stride=64, y_token_stride=64, cu=_at(7), total=T, longest=0, batch=2, C=C, G=G, reverse=0, dtype=BF16)
    a.update(change)
    return eq.RecurrenceArgs(**a)


@pytest.mark.parametrize("change, want", [
    (dict(dtype=3), INVALID), (dict(total=-1), INVALID), (dict(batch=-1), INVALID), (dict(longest=-1), INVALID), (dict(C=0), INVALID),
    (dict(G=3), INVALID), (dict(C=1 << 19), UNSUPPORTED), (dict(total=(1 << 30) + 1), UNSUPPORTED), (dict(batch=(1 << 24) + 1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(forget=None), INVALID), (dict(y=None), INVALID), (dict(cu=None), INVALID), (dict(x=_at(0) + 1), INVALID),
    (dict(y=_at(3) + 1), INVALID), (dict(cu=_at(7) + 2), INVALID), (dict(state=_at(4) + 2), INVALID), (dict(final=_at(5) + 1), INVALID),
    (dict(marks=_at(6) + 2), INVALID), (dict(x_token_stride=-64), INVALID), (dict(forget_token_stride=63), INVALID), (dict(gate_token_stride=0), INVALID), (dict(y_token_stride=63), INVALID), (dict(y_token_stride=0), INVALID),
    (dict(gate_token_stride=(1 << 24) + 1), INVALID), (dict(y=_at(0)), INVALID), (dict(y=_at(2) + 64), INVALID), (dict(final=_at(4) + 64), INVALID),
    (dict(final=_at(1)), INVALID), (dict(marks=_at(4)), INVALID), (dict(marks=_at(5)), INVALID), (dict(y=_at(7) - 4096), INVALID),
    (dict(marks=_at(7)), INVALID), (dict(total=10000, batch=1), INVALID)])
def test_recurrence_refusals(lib, change, want):  # noqa: F811
    a = _rec(**change)
    _refused(lib, lib.eqlin_recurrence(ctypes.byref(a), None, 0, None), want)


def test_recurrence_of_nothing_and_sizes(lib):  # noqa: F811
    assert lib.eqlin_recurrence(ctypes.byref(_rec(batch=0, x=None, cu=None)), None, 0, None) == 0
    _refused(lib, lib.eqlin_recurrence(None, None, 0, None), INVALID)
    assert lib.eqlin_recurrence_workspace(None) == 0 and lib.eqlin_recurrence_workspace(ctypes.byref(_rec(G=5))) == 0
    assert lib.eqlin_recurrence_marks(0, 3) == 3 and lib.eqlin_recurrence_marks(1000, 2) == 17 and lib.eqlin_recurrence_marks(-1, 2) == 0
    assert lib.eqlin_recurrence_workspace(ctypes.byref(_rec(total=1 << 20, longest=100))) == 0  # a sequence a workgroup
    slots = (1 << 20) // 64 + 2
    assert lib.eqlin_recurrence_workspace(ctypes.byref(_rec(total=1 << 20))) == 12 * slots * 64  # one that may be long


@pytest.mark.parametrize("change", [
    dict(dy=None), dict(dx=None), dict(dforget=None), dict(dx=_at(0)), dict(dx=_at(8)), dict(dforget=_at(10) + 64), dict(dgate=_at(10) + 32),
    dict(dstate=_at(9)), dict(dstate=_at(9) + 64), dict(dstate=_at(10) + 64), dict(dx=_at(6)), dict(dx_token_stride=32), dict(dy=_at(8) + 1),
    dict(dx=_at(11) + 64, dx_token_stride=96), dict(dfinal=_at(9) + 2), dict(dx=_at(7))])
def test_recurrence_backward_refusals(lib, change):  # noqa: F811
    g = dict(dy=_at(8), dfinal=_at(9), dx=_at(10), dforget=_at(11), dgate=_at(12), dstate=_at(13), dy_token_stride=64, dx_token_stride=64,
             dforget_token_stride=64, dgate_token_stride=64)
    a, grads = _rec(), eq.RecurrenceGrads(**{**g, **change})
    _refused(lib, lib.eqlin_recurrence_backward(ctypes.byref(a), ctypes.byref(grads), None, 0, None), INVALID)


def test_recurrence_backward_refuses_what_it_lacks(lib):  # noqa: F811
    g = eq.RecurrenceGrads(dy=_at(8), dx=_at(10), dforget=_at(11), dgate=_at(12), dy_token_stride=64, dx_token_stride=64, dforget_token_stride=64,
                           dgate_token_stride=64)
    for change in (dict(marks=None), dict(gate=None), dict(cu=None)):
        _refused(lib, lib.eqlin_recurrence_backward(ctypes.byref(_rec(**change)), ctypes.byref(g), None, 0, None), INVALID)
    _refused(lib, lib.eqlin_recurrence_backward(ctypes.byref(_rec()), None, None, 0, None), INVALID)
