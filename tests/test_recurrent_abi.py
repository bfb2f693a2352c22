"""Host-side argument checks of the recurrent stage's C entry points: each wrong argument gives its status and a message, before
anything touches a GPU (the pointers here are never followed)."""
import pytest

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
