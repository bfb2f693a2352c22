"""Host-side checks that no memory which a stage operator writes is written twice or read as an input: outputs whose strides
fold them onto themselves, the index arrays, lse, the workspace, and gradients that share elements. The pointers here are
never followed: every call is refused, and what a test wants to see accepted is refused by a later check."""
import ctypes
import random

import pytest

import fourier_domain_linear_amd as eq
from test_stage_abi import BF16, INVALID, _args, _at, _norm


@pytest.fixture(scope="module")
def lib():
    return eq.load_library()


def _message(lib, status):
    assert status == INVALID, lib.eqlin_last_error().decode()
    return lib.eqlin_last_error().decode()


def _elements(ts, hs, tokens, heads, dim):
    return [i * ts + j * hs + e for i in range(tokens) for j in range(heads) for e in range(dim)]


def test_strides_that_fold(lib):
    """All strides up to 40 at random, against every element's place."""
    rng, seen = random.Random(1), set()
    for _ in range(4000):
        N, H, D, ts, hs = rng.randint(1, 6), rng.randint(1, 6), rng.randint(2, 5), rng.randint(0, 40), rng.randint(0, 40)
        at = _elements(ts, hs, N, H, D)
        fold = len(set(at)) < len(at)
        # where y does not fold, x in its last element is refused
        said = _message(lib, lib.eqlin_rotary(_at(0) + 2 * max(at), D, 0, _at(0), ts, hs, _at(1), N, H, D, 1, 1, (ctypes.c_int * 1)(1),
                                              100.0, 0, BF16, None))
        assert said == ("y's strides fold it onto itself" if fold else "x and y overlap"), (N, H, D, ts, hs, said)
        seen.add((fold, hs >= D and ts >= D and N > 1 and H > 1 and ts < (H - 1) * hs + D and hs < (N - 1) * ts + D))
    assert len(seen) == 4  # (both answers among the interleaved strides)


def test_strides_that_fold_are_quick_to_check(lib):
    """A million tokens and heads of strides that need the long way."""
    said = _message(lib, lib.eqlin_rotary(_at(0) + 64, 8, 0, _at(0), (1 << 21) + 16, 24, _at(1), 1 << 30, 1 << 20, 8, 1, 1, (ctypes.c_int * 1)(1),
                                          100.0, 0, BF16, None))
    assert said in ("y's strides fold it onto itself", "x and y overlap")


@pytest.mark.parametrize("strides", [(64, 128), (128, 64 * 3), (192, 128)])
def test_attention_output_that_folds(lib, strides):
    a = _args(o_token_stride=strides[0], o_head_stride=strides[1])
    assert "fold" in _message(lib, lib.eqlin_attention(ctypes.byref(a), None, 0, None))


def _grads(**change):
    g = dict(d_o=_at(7), dq=_at(8), dk=_at(9), dv=_at(10), do_token_stride=256, do_head_stride=64, dq_token_stride=256, dq_head_stride=64,
             dk_token_stride=128, dk_head_stride=64, dv_token_stride=128, dv_head_stride=64)
    g.update(change)
    return eq.AttentionGrads(**g)


@pytest.mark.parametrize("name", ["cu_q", "cu_k", "len_k"])
@pytest.mark.parametrize("over", ["o", "lse"])
def test_attention_results_over_the_bounds(lib, name, over):
    a = _args(len_k=_at(12))
    setattr(a, name, getattr(a, over) + 16)
    assert _message(lib, lib.eqlin_attention(ctypes.byref(a), _at(11), 1 << 30, None)) == f"{over} overlaps the input {name}"


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "lse", "cu_q", "cu_k", "len_k"])
def test_attention_workspace_over_a_tensor(lib, name):
    a = _args(total_k=4000, cu_q=_at(5), len_k=_at(12))  # one token run over many keys: a workspace
    need = lib.eqlin_attention_workspace(ctypes.byref(a))
    assert need > 0
    said = _message(lib, lib.eqlin_attention(ctypes.byref(a), getattr(a, name) - need + 256 & ~255, need, None))
    assert "workspace" in said and said.endswith(name), said


@pytest.mark.parametrize("name", ["cu_q", "cu_k", "len_k", "lse", "q", "k", "v", "o"])
@pytest.mark.parametrize("over", ["dq", "dk", "dv"])
def test_attention_gradients_over_an_input(lib, name, over):
    a, g = _args(len_k=_at(12)), _grads()
    setattr(a, name, getattr(g, over) + 16)
    assert _message(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(g), _at(11), 1 << 30, None)) == f"{over} overlaps the input {name}"


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "lse", "cu_q", "cu_k", "len_k", "d_o", "dq", "dk", "dv"])
def test_attention_backward_workspace_over_a_tensor(lib, name):
    a, g = _args(len_k=_at(12)), _grads()
    at = getattr(a, name, None) or getattr(g, name)
    said = _message(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(g), at, 1 << 30, None))
    assert "workspace" in said and said.endswith(name), said


def test_gradients_that_share_elements(lib):
    """dk and dv of one layout, one behind the other by any distance, against every element's place. (Where they are apart, dv's
    end over cu_k is refused.)"""
    rng, seen = random.Random(2), set()
    for _ in range(3000):
        T, H, D = rng.randint(1, 5), rng.choice([1, 2, 4]), rng.choice([8, 16])
        ts, hs, by = 8 * rng.randint(1, 20), 8 * rng.randint(1, 20), 8 * rng.randint(1, 60)
        at = _elements(ts, hs, T, H, D)
        if len(set(at)) < len(at):
            continue
        meet = bool(set(at) & {e + by for e in at})
        a = _args(total_k=T, heads_kv=H, dim=D, k_token_stride=H * D, k_head_stride=D, v_token_stride=H * D, v_head_stride=D,
                  cu_k=_at(9) + 2 * (by + max(at)) - 6)
        g = _grads(dv=_at(9) + 2 * by, dk_token_stride=ts, dk_head_stride=hs, dv_token_stride=ts, dv_head_stride=hs)
        said = _message(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(g), _at(11), 1 << 30, None))
        assert said == ("dk and dv share memory" if meet else "dv overlaps the input cu_k"), (T, H, D, ts, hs, by, said)
        seen.add(meet)
    assert len(seen) == 2


def test_gradients_of_one_head_or_token_that_share_elements(lib):
    """A stride over one head or token means nothing, so the other tensor's decides."""
    a = _args(heads_q=4, heads_kv=1)
    g = _grads(dk=_at(8) + 2 * (64 + 8), dq_token_stride=512, dk_token_stride=512)  # dk in dq's second and third head
    assert _message(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(g), _at(11), 1 << 30, None)) == "dq and dk share memory"
    a = _args(total_q=1)
    g = _grads(dk=_at(8) + 2 * 64)  # dk's first heads in dq's only token
    assert _message(lib, lib.eqlin_attention_backward(ctypes.byref(a), ctypes.byref(g), _at(11), 1 << 30, None)) == "dq and dk share memory"


def test_norm_backward_memory_that_is_shared(lib):
    args = [_at(0), _at(1), _at(2), _at(3), _at(4), _at(5), _at(6)]  # sum, gamma, rstd, dy, dsum, dx, dgamma
    for i, name in enumerate(["sum", "gamma", "rstd", "dy", "dsum", "dx", "dgamma"]):
        said = _message(lib, lib.eqlin_rmsnorm_backward(*args, 8, 16, 4, BF16, args[i], 1 << 20, None))
        assert "workspace" in said and said.endswith(name), said
    assert _message(lib, _norm(lib, y=_at(1))) == "y overlaps the input residual"
