"""Pins of oracle/stage.py (norm, rotary positions, attention and their gradients) against things other than
itself: central differences, closed forms, equivariance under the group, and the e4m3 format's definition."""
import numpy as np
import pytest
import torch

from oracle import stage


def _rng(seed):
    return np.random.default_rng(seed)


def _diff(f, x, h=1e-5):
    """Central differences of a scalar f at x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        g[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


def test_rmsnorm_closed_forms():
    x = np.full((2, 3, 4), 2.0)
    y, s, rstd = stage.rmsnorm(x, eps=0.0)
    assert np.allclose(y, 1) and np.allclose(rstd, 0.5) and np.array_equal(s, x)
    y, s, _ = stage.rmsnorm(x, gamma=np.array([1.0, -2.0, 0.0]), residual=-x)
    assert not s.any() and not y.any()
    x = _rng(0).standard_normal((5, 6, 2))
    y, _, rstd = stage.rmsnorm(x, eps=0.0)
    assert np.allclose((y ** 2).mean(axis=(1, 2)), 1)
    assert np.allclose(stage.rmsnorm(7 * x, eps=0.0)[0], y)


def test_e4m3_format():
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    fine = codes[np.isfinite(codes)]
    assert set(np.abs(fine)) == set(stage._E4M3) and stage._E4M3[-1] == 448
    assert np.array_equal(stage.e4m3_nearest(fine), fine)
    v = _rng(1).standard_normal(4000) * 100
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(stage.e4m3_nearest(v.astype(np.float32)), want)


@pytest.mark.parametrize("G", [1, 4])
def test_rmsnorm_gradients(G):
    r = _rng(2)
    x, dy, ds, g = r.standard_normal((3, 4, G)), r.standard_normal((3, 4, G)), r.standard_normal((3, 4, G)), r.standard_normal(4)
    loss = lambda a, b: (stage.rmsnorm(a, b)[0] * dy).sum() + (a * ds).sum()  # noqa: E731
    dx, dg = stage.rmsnorm_backward(dy, x, g, stage.rmsnorm(x, g)[2], ds)
    assert np.allclose(dx, _diff(lambda a: loss(a, g), x), atol=1e-8)
    assert np.allclose(dg, _diff(lambda b: loss(x, b), g), atol=1e-8)


def test_rotary_closed_forms():
    x = _rng(3).standard_normal((2, 1, 5, 1))
    assert np.allclose(stage.rotary(x, [[0], [0]], [2]), x)
    y = stage.rotary(np.array([1.0, 0, 0, 0, 9]).reshape(1, 1, 5, 1), [[3]], [2], base=100.0)[0, 0, :, 0]
    assert np.allclose(y, [np.cos(3), 0, np.sin(3), 0, 9])
    y = stage.rotary(np.array([0, 1.0, 0, 0, 9]).reshape(1, 1, 5, 1), [[3]], [2], base=100.0)[0, 0, :, 0]
    assert np.allclose(y, [0, np.cos(0.3), 0, np.sin(0.3), 9])
    pos = _rng(4).integers(0, 50, (6, 3))
    x = _rng(5).standard_normal((6, 2, 8, 4))
    y = stage.rotary(x, pos, [1, 1, 2])
    assert np.allclose(stage.rotary(y, pos, [1, 1, 2], inverse=True), x)
    dy = _rng(6).standard_normal(x.shape)  # the inverse is the adjoint
    assert np.isclose((y * dy).sum(), (x * stage.rotary(dy, pos, [1, 1, 2], inverse=True)).sum())


def test_rotary_scores_depend_on_differences():
    r = _rng(7)
    q, k = r.standard_normal((1, 1, 8, 1)), r.standard_normal((1, 1, 8, 1))
    a = (stage.rotary(q, [[5, 9]], [2, 2]) * stage.rotary(k, [[2, 11]], [2, 2])).sum()
    b = (stage.rotary(q, [[15, 4]], [2, 2]) * stage.rotary(k, [[12, 6]], [2, 2])).sum()
    assert np.isclose(a, b)


@pytest.mark.parametrize("d4", [False, True], ids=["p4", "d4"])
def test_rotary_commutes_with_the_group(d4):
    """x'[h p, g] = x[p, h^-1 g] (turned or mirrored image, shifted group axis): the operator commutes."""
    r, G = _rng(8), 8 if d4 else 4
    x, pos = r.standard_normal((5, 2, 8, G)), r.integers(-7, 8, (5, 3))
    els = [(a, b) for b in range(2 if d4 else 1) for a in range(4)]
    R, S = np.array([[0, -1], [1, 0]]), np.diag([1, -1])
    mat = lambda e: np.linalg.matrix_power(R, e[0]) @ (S if e[1] else np.eye(2, dtype=int))  # noqa: E731
    index = lambda m: next(i for i, e in enumerate(els) if np.array_equal(mat(e), m))  # noqa: E731
    y = stage.rotary(x, pos, [1, 1, 2], d4=d4)
    for h in els:
        inv = np.rint(np.linalg.inv(mat(h))).astype(int)
        perm = [index(inv @ mat(g)) for g in els]
        pos2 = pos.copy()
        pos2[:, 1:] = pos[:, 1:] @ mat(h).T
        assert np.allclose(stage.rotary(x[..., perm], pos2, [1, 1, 2], d4=d4), y[..., perm])


def test_attention_closed_forms():
    r = _rng(9)
    v = r.standard_normal((6, 1, 4))
    k = r.standard_normal((6, 1, 4))
    o, lse = stage.attention(np.zeros((3, 2, 4)), k, v, [0, 1, 3], [0, 4, 6])
    assert np.allclose(o[0, 1], v[:4, 0].mean(0)) and np.allclose(o[1:, 0], v[4:, 0].mean(0))
    assert np.allclose(lse[0], np.log(4)) and np.allclose(lse[1:], np.log(2))
    o, lse = stage.attention(np.zeros((3, 2, 4)), k, v, [0, 1, 3], [0, 4, 6], causal=True, len_k=[2, 1])
    assert np.allclose(o[0, 0], v[:2, 0].mean(0)) and not o[1].any() and np.allclose(o[2, 1], v[4, 0])
    assert np.isneginf(lse[1]).all()
    k[1] = np.nan  # a key that nobody sees
    v[1] = np.inf
    o, _ = stage.attention(r.standard_normal((1, 2, 4)), k, v, [0, 1], [0, 6], len_k=[1])
    assert np.allclose(o, v[0])


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradients(causal):
    r = _rng(10)
    q, k, v, do = r.standard_normal((5, 4, 3)), r.standard_normal((6, 2, 3)), r.standard_normal((6, 2, 3)), r.standard_normal((5, 4, 3))
    cu_q, cu_k, len_k = [0, 3, 5], [0, 2, 6], [2, 3]
    f = lambda a, b, c: (stage.attention(a, b, c, cu_q, cu_k, causal, 0.7, len_k)[0] * do).sum()  # noqa: E731
    dq, dk, dv = stage.attention_backward(do, q, k, v, cu_q, cu_k, causal, 0.7, len_k)
    assert np.allclose(dq, _diff(lambda a: f(a, k, v), q), atol=1e-8)
    assert np.allclose(dk, _diff(lambda a: f(q, a, v), k), atol=1e-8)
    assert np.allclose(dv, _diff(lambda a: f(q, k, a), v), atol=1e-8)


def test_attention_follows_a_shift_of_the_group_axis():
    r = _rng(11)
    q, k, v = (r.standard_normal((5, 2, 3, 4)) for _ in range(3))
    run = lambda *t: stage.attention(*(a.reshape(5, 2, 12) for a in t), [0, 5], [0, 5])[0].reshape(5, 2, 3, 4)  # noqa: E731
    assert np.allclose(run(*(np.roll(t, 1, axis=3) for t in (q, k, v))), np.roll(run(q, k, v), 1, axis=3))
