"""Host-side argument checks of the stage operators' C entry points: each wrong argument gives its status and a message,
before anything touches a GPU (the pointers here are never followed)."""
import ctypes

import pytest

import fourier_domain_linear_amd as eq

P = 1 << 20  # a pointer's stand-in, aligned
INVALID, UNSUPPORTED = 1, 2
BF16 = 1


@pytest.fixture(scope="module")
def lib():
    return eq.load_library()


def _at(i):
    return P + (i << 40)


def _refused(lib, status, want):
    assert status == want, lib.eqlin_last_error().decode()
    assert lib.eqlin_last_error().decode()


def _norm(lib, x=_at(0), residual=_at(1), gamma=_at(2), s=_at(3), y=_at(4), rstd=_at(5), N=8, C=16, G=4, eps=1e-6, dtype=BF16):
    return lib.eqlin_rmsnorm(x, residual, gamma, s, y, rstd, N, C, G, eps, dtype, None)


@pytest.mark.parametrize("change, want", [
    (dict(N=-1), INVALID), (dict(C=0), INVALID), (dict(G=3), INVALID), (dict(dtype=7), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x=_at(0) + 2), INVALID), (dict(y=_at(0)), INVALID), (dict(s=_at(4) + 16), INVALID), (dict(rstd=_at(5) + 1), INVALID),
    (dict(C=1 << 20), UNSUPPORTED), (dict(N=1 << 60), INVALID)])
def test_norm_refusals(lib, change, want):
    _refused(lib, _norm(lib, **change), want)


def test_norm_of_nothing(lib):
    assert _norm(lib, N=0, x=None, y=None) == 0
    assert lib.eqlin_rmsnorm_backward_workspace(0, 16, 4) == 0


def test_norm_backward_needs_its_workspace(lib):
    _refused(lib, lib.eqlin_rmsnorm_backward(_at(0), _at(1), _at(2), _at(3), _at(4), _at(5), _at(6), 8, 16, 4, BF16, None, 0, None), INVALID)
    _refused(lib, lib.eqlin_rmsnorm_backward(_at(0), _at(1), _at(2), _at(3), _at(4), _at(0), None, 8, 16, 4, BF16, None, 0, None), INVALID)


def _rotary(lib, x=_at(0), y=_at(1), pos=_at(2), xt=512, xh=64, yt=512, yh=64, N=10, H=8, dc=16, G=4, axes=2, pairs=(4, 4),
            base=10000.0, flags=0, dtype=BF16):
    p = (ctypes.c_int * max(1, len(pairs)))(*pairs)
    return lib.eqlin_rotary(x, xt, xh, y, yt, yh, pos, N, H, dc, G, axes, p, base, flags, dtype, None)


@pytest.mark.parametrize("change, want", [
    (dict(dtype=9), INVALID), (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(G=5), INVALID), (dict(flags=2), INVALID),
    (dict(flags=4), INVALID), (dict(axes=0, pairs=()), INVALID), (dict(axes=5, pairs=(1,) * 5), INVALID), (dict(pairs=(5, 4)), INVALID),
    (dict(pairs=(0, 0)), INVALID), (dict(pairs=(-1, 4)), INVALID), (dict(base=0.0), INVALID), (dict(base=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(x=_at(0) + 1), INVALID), (dict(yh=32), INVALID), (dict(yt=0), INVALID),
    (dict(xt=-512), INVALID), (dict(y=_at(0) + 64), INVALID), (dict(y=_at(0), yt=1024), INVALID), (dict(pos=_at(1)), INVALID),
    (dict(N=1 << 34, xt=1 << 24, yt=1 << 24), UNSUPPORTED), (dict(H=1 << 21), UNSUPPORTED)])
def test_rotary_refusals(lib, change, want):
    _refused(lib, _rotary(lib, **change), want)


def _args(**change):
    T, S, Hq, Hkv, D = 10, 12, 4, 2, 64
    a = dict(q=_at(0), k=_at(1), v=_at(2), o=_at(3), lse=_at(4), q_token_stride=Hq * D, q_head_stride=D, k_token_stride=Hkv * D,
             k_head_stride=D, v_token_stride=Hkv * D, v_head_stride=D, o_token_stride=Hq * D, o_head_stride=D, cu_q=_at(5), cu_k=_at(6),
             len_k=None, total_q=T, total_k=S, batch=1, heads_q=Hq, heads_kv=Hkv, dim=D, scale=0.125, causal=0, dtype=BF16)
    a.update(change)
    return eq.AttentionArgs(**a)


@pytest.mark.parametrize("change, want", [
    (dict(dtype=3), INVALID), (dict(batch=-1), INVALID), (dict(total_q=-1), INVALID), (dict(heads_q=3), INVALID), (dict(heads_kv=0), INVALID),
    (dict(dim=0), INVALID), (dict(dim=136), UNSUPPORTED), (dict(dim=12), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(total_q=1 << 28), UNSUPPORTED), (dict(batch=1 << 21), UNSUPPORTED), (dict(q=None), INVALID), (dict(v=None), INVALID),
    (dict(k=_at(1) + 8), INVALID), (dict(k_token_stride=129), INVALID), (dict(k_token_stride=-128), INVALID),
    (dict(k_token_stride=1 << 24), UNSUPPORTED), (dict(k_head_stride=1 << 62), UNSUPPORTED), (dict(q_head_stride=1 << 27), UNSUPPORTED),
    (dict(o_head_stride=32), INVALID), (dict(o_token_stride=0), INVALID), (dict(cu_q=None), INVALID), (dict(cu_k=_at(6) + 2), INVALID)])
def test_attention_refusals(lib, change, want):
    a = _args(**change)
    _refused(lib, lib.eqlin_attention(ctypes.byref(a), None, 0, None), want)


def test_attention_of_nothing(lib):
    for change in (dict(total_q=0, q=None, o=None), dict(batch=0, q=None)):
        a = _args(**change)
        assert lib.eqlin_attention(ctypes.byref(a), None, 0, None) == 0
    _refused(lib, lib.eqlin_attention(None, None, 0, None), INVALID)
    assert lib.eqlin_attention_workspace(ctypes.byref(_args(dim=12))) == 0


def test_attention_backward_refusals(lib):
    g = dict(d_o=_at(7), dq=_at(8), dk=_at(9), dv=_at(10), do_token_stride=256, do_head_stride=64, dq_token_stride=256, dq_head_stride=64,
             dk_token_stride=128, dk_head_stride=64, dv_token_stride=128, dv_head_stride=64)
    a = _args()
    for change in (dict(d_o=None), dict(dq=None), dict(dk_token_stride=8), dict(dv_head_stride=0), dict(dk=_at(10)), dict(dq=_at(9))):
        grads = eq.AttentionGrads(**{**g, **change})
        _refused(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(grads), _at(11), 1 << 30, None), INVALID)
    _refused(lib, lib.eqlin_attention_backward(ctypes.byref(a), None, _at(11), 1 << 30, None), INVALID)
    none = _args(lse=None)
    grads = eq.AttentionGrads(**g)
    _refused(lib, lib.eqlin_attention_backward(ctypes.byref(none), ctypes.byref(grads), _at(11), 1 << 30, None), INVALID)
