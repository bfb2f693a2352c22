"""Pins of the recurrent stage's part of oracle/stage.py (layer norm, gated recurrence and their gradients) against things
other than itself: closed forms, central differences, equivariance, and mistakes planted in the formulas."""
import numpy as np
import pytest

from oracle import stage
from test_oracle_stage import _diff, _rng


def test_layernorm_closed_forms():
    x = np.zeros((2, 2, 2))
    x[:, 0], x[:, 1] = 5.0, 1.0
    y, s, mean, rstd = stage.layernorm(x, eps=0.0)
    assert np.allclose(mean, 3) and np.allclose(rstd, 0.5) and np.allclose(y[:, 0], 1) and np.allclose(y[:, 1], -1)
    y, s, _, _ = stage.layernorm(x, gamma=np.array([2.0, 0.0]), beta=np.array([1.0, 7.0]), residual=x)
    assert np.array_equal(s, 2 * x) and np.allclose(y[:, 1], 7) and np.allclose(y[:, 0], 3, atol=1e-5)
    x = _rng(0).standard_normal((5, 6, 2))
    y, _, _, _ = stage.layernorm(x, eps=0.0)
    assert np.allclose(y.mean(axis=(1, 2)), 0) and np.allclose((y ** 2).mean(axis=(1, 2)), 1)
    assert np.allclose(stage.layernorm(7 * x + 100, eps=0.0)[0], y)
    assert np.allclose(stage.layernorm(np.roll(x, 1, 2), eps=0.0)[0], np.roll(y, 1, 2))


@pytest.mark.parametrize("G", [1, 4])
def test_layernorm_gradients(G):
    r = _rng(1)
    x, dy, ds = (r.standard_normal((3, 4, G)) for _ in range(3))
    g, b = r.standard_normal(4), r.standard_normal(4)
    loss = lambda a, c, d: (stage.layernorm(a, c, d)[0] * dy).sum() + (a * ds).sum()  # noqa: E731
    _, _, mean, rstd = stage.layernorm(x, g, b)
    dx, dg, db = stage.layernorm_backward(dy, x, g, mean, rstd, ds)
    assert np.allclose(dx, _diff(lambda a: loss(a, g, b), x), atol=1e-8)
    assert np.allclose(dg, _diff(lambda a: loss(x, a, b), g), atol=1e-8)
    assert np.allclose(db, _diff(lambda a: loss(x, g, a), b), atol=1e-8)


def test_recurrence_closed_forms():
    x, z = np.ones((4, 1, 1)), np.zeros((4, 1, 1))
    y, final, _ = stage.recurrence(x, z, [0, 3, 3, 4], state=np.array([0.0, 5.0, 3.0]).reshape(3, 1, 1))
    assert np.allclose(y.ravel(), [0.5, 0.75, 0.875, 2.0]) and np.allclose(final.ravel(), [0.875, 5, 2])
    y, final, _ = stage.recurrence(x, z, [0, 3, 4], reverse=True)
    assert np.allclose(y.ravel(), [0.875, 0.75, 0.5, 0.5]) and np.allclose(final.ravel(), [0.875, 0.5])
    far = np.full((4, 1, 1), 40.0)
    assert np.allclose(stage.recurrence(x, far, [0, 4], state=np.full((1, 1, 1), 9.0))[0], 9)  # nothing forgotten
    assert np.allclose(stage.recurrence(x, -far, [0, 4], state=np.full((1, 1, 1), 9.0))[0], 1)  # all of it
    o = np.array([0.0, 100.0, -100.0, np.log(3.0)]).reshape(4, 1, 1)
    y, _, h = stage.recurrence(x, z, [0, 4], gate=o)
    assert np.allclose(y.ravel(), [0, 100 * h[1, 0, 0], 0, h[3, 0, 0] * 0.75 * np.log(3.0)])
    y, _, _ = stage.recurrence(x, z, [1, 3])
    assert np.isnan(y[[0, 3]]).all() and np.allclose(y[1:3].ravel(), [0.5, 0.75])


def _case(seed=2):
    r = _rng(seed)
    x, z, o, dy = (r.standard_normal((7, 2, 2)) for _ in range(4))
    return x, z, o, dy, r.standard_normal((4, 2, 2)), r.standard_normal((4, 2, 2)), [0, 3, 3, 4, 7]


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_recurrence_gradients(gated, reverse):
    x, z, o, dy, h0, df, cu = _case()
    o = o if gated else None

    def loss(a, b, c, h):
        y, final, _ = stage.recurrence(a, b, cu, c, h, reverse)
        return (y * dy).sum() + (final * df).sum()

    dx, dz, do, dh = stage.recurrence_backward(dy, x, z, cu, o, h0, reverse, df)
    assert np.allclose(dx, _diff(lambda a: loss(a, z, o, h0), x), atol=1e-8)
    assert np.allclose(dz, _diff(lambda a: loss(x, a, o, h0), z), atol=1e-8)
    assert np.allclose(dh, _diff(lambda a: loss(x, z, o, a), h0), atol=1e-8)
    if gated:
        assert np.allclose(do, _diff(lambda a: loss(x, z, a, h0), o), atol=1e-8)


def test_recurrence_in_pieces_and_under_a_shift_of_the_group_axis():
    x, z, o, _, h0, _, _ = _case(3)
    whole, final, _ = stage.recurrence(x, z, [0, 7], o, h0[:1])
    a, mid, _ = stage.recurrence(x[:4], z[:4], [0, 4], o[:4], h0[:1])
    b, end, _ = stage.recurrence(x[4:], z[4:], [0, 3], o[4:], mid)
    assert np.allclose(np.concatenate([a, b]), whole) and np.allclose(end, final)
    roll = lambda t: np.roll(t, 1, 2)  # noqa: E731
    assert np.allclose(stage.recurrence(roll(x), roll(z), [0, 7], roll(o), roll(h0[:1]))[0], roll(whole))


@pytest.mark.parametrize("slip", ["sequence's end", "token order", "state lost", "gate's slope", "forget's slope"])
def test_planted_mistakes_are_seen(slip):
    """The closed forms and differences above tell each of these from the definition."""
    x, z, o, dy, h0, df, cu = _case(4)
    y, final, _ = stage.recurrence(x, z, cu, o, h0)
    dx, dz, do, _ = stage.recurrence_backward(dy, x, z, cu, o, h0, False, df)
    if slip == "sequence's end":
        assert not np.allclose(stage.recurrence(x, z, [0, 7, 7, 7, 7], o, h0)[0], y)
    elif slip == "token order":
        assert not np.allclose(stage.recurrence(x, z, cu, o, h0, reverse=True)[0], y)
    elif slip == "state lost":
        assert not np.allclose(stage.recurrence(x, z, cu, o)[1], final)
    elif slip == "gate's slope":  # silu's derivative without its second term
        sig = 1 / (1 + np.exp(-o))
        assert not np.allclose(dy * stage.recurrence(x, z, cu, None, h0)[0] * sig, do)
    else:  # the share of x left out of the gate's gradient
        assert not np.allclose(dz, dz + dx * x / (1 + np.exp(-z)))


@pytest.mark.parametrize("slip", ["x left out", "state of the token itself", "the gate's own factor left out"])
def test_slips_in_the_forget_gates_gradient_are_seen(slip):
    """dforget = dh (h[t-1] - x) f (1 - f): central differences agree with it and with none of the slips."""
    x, z, o, dy, h0, df, cu = _case(5)
    dx, dz, _, _ = stage.recurrence_backward(dy, x, z, cu, o, h0, False, df)

    def loss(b):
        y, final, _ = stage.recurrence(x, b, cu, o, h0)
        return (y * dy).sum() + (final * df).sum()

    want = _diff(loss, z)
    f, keep = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    dh = dx / keep
    h = stage.recurrence(x, z, cu, None, h0)[0]
    before = np.concatenate([h[:1], h[:-1]])
    for i in range(4):
        if cu[i] < cu[i + 1]:
            before[cu[i]] = h0[i]
    assert np.allclose(dz, want, atol=1e-8) and np.allclose(dh * (before - x) * f * keep, want, atol=1e-8)
    wrong = {"x left out": dh * before * f * keep, "state of the token itself": dh * (h - x) * f * keep,
             "the gate's own factor left out": dh * (before - x) * keep}[slip]
    assert not np.allclose(wrong, want, atol=1e-3)
