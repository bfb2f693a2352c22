"""fp64 CPU oracle of the operators between the layers of a transformer or recurrent stage: root-mean-square and layer norm
with the residual's addition, rotary positions over several axes, attention and the gated recurrence over packed sequences,
and their gradients.

TEST INFRASTRUCTURE ONLY, written from the formulas in plain numpy loops over tokens' sequences and heads; it
shares no code with the GPU path. Pinned in ``tests/test_oracle_stage.py`` against central differences,
closed forms, and the group's equivariance.
"""
from __future__ import annotations

import numpy as np

# e4m3 (OCP): the 127 non-negative finite values, for the nearest-even rounding of rmsnorm_quant
_E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8) if not (e == 15 and m == 7)])


def rmsnorm(x, gamma=None, residual=None, eps=1e-6):
    """(y, s, rstd) of x [N, C, G]."""
    s = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1 / np.sqrt((s ** 2).mean(axis=(1, 2)) + eps)
    g = np.ones(s.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    return s * rstd[:, None, None] * g[None, :, None], s, rstd


def e4m3_nearest(v):
    """v rounded to the nearest e4m3 value, ties to the even code; beyond the largest, the largest."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), _E4M3[-1])
    hi = np.clip(np.searchsorted(_E4M3, a), 1, len(_E4M3) - 1)
    lo = hi - 1
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(_E4M3[code], v)


def rmsnorm_quant(x, gamma=None, residual=None, eps=1e-6):
    """(q, scale, s, rstd): q the e4m3 values."""
    y, s, rstd = rmsnorm(x, gamma, residual, eps)
    amax = np.abs(y).max(axis=(1, 2))
    scale = np.where(amax > 0, amax / 448, 1.0)
    return e4m3_nearest(y / scale[:, None, None]), scale, s, rstd


def rmsnorm_backward(dy, s, gamma, rstd, ds=None):
    """(dx, dgamma) with s and rstd as given."""
    dy, s, rstd = (np.asarray(t, np.float64) for t in (dy, s, rstd))
    g = np.ones(s.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    xh = s * rstd[:, None, None]
    w = dy * g[None, :, None]
    dx = rstd[:, None, None] * (w - xh * (w * xh).mean(axis=(1, 2))[:, None, None])
    return dx + (0 if ds is None else np.asarray(ds, np.float64)), (dy * xh).sum(axis=(0, 2))


def layernorm(x, gamma=None, beta=None, residual=None, eps=1e-5):
    """(y, s, mean, rstd) of x [N, C, G]."""
    s = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    mean = s.mean(axis=(1, 2))
    d = s - mean[:, None, None]
    rstd = 1 / np.sqrt((d ** 2).mean(axis=(1, 2)) + eps)
    g = np.ones(s.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    b = np.zeros(s.shape[1]) if beta is None else np.asarray(beta, np.float64)
    return d * rstd[:, None, None] * g[None, :, None] + b[None, :, None], s, mean, rstd


def layernorm_backward(dy, s, gamma, mean, rstd, ds=None):
    """(dx, dgamma, dbeta) with s, mean and rstd as given."""
    dy, s, mean, rstd = (np.asarray(t, np.float64) for t in (dy, s, mean, rstd))
    g = np.ones(s.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    xh = (s - mean[:, None, None]) * rstd[:, None, None]
    w = dy * g[None, :, None]
    dx = rstd[:, None, None] * (w - w.mean(axis=(1, 2))[:, None, None] - xh * (w * xh).mean(axis=(1, 2))[:, None, None])
    return dx + (0 if ds is None else np.asarray(ds, np.float64)), (dy * xh).sum(axis=(0, 2)), dy.sum(axis=(0, 2))


def _runs(cu, reverse):
    """The tokens of each sequence in the recurrence's order."""
    for i in range(len(cu) - 1):
        t = list(range(cu[i], cu[i + 1]))
        yield t[::-1] if reverse else t


def recurrence(x, forget, cu, gate=None, state=None, reverse=False):
    """(y, final, h) of h_t = f h_{t-1} + (1 - f) x_t, f = sigmoid(forget), y = h or h silu(gate). x [T, C, G]; rows outside
    every sequence are NaN in y and h."""
    x, z = np.asarray(x, np.float64), np.asarray(forget, np.float64)
    h = np.full(x.shape, np.nan)
    final = np.zeros((len(cu) - 1,) + x.shape[1:]) if state is None else np.array(state, np.float64)
    for i, run in enumerate(_runs(cu, reverse)):
        for t in run:
            f = 1 / (1 + np.exp(-z[t]))
            final[i] = f * final[i] + x[t] / (1 + np.exp(z[t]))
            h[t] = final[i]
    if gate is None:
        return h, final, h
    o = np.asarray(gate, np.float64)
    return h * o / (1 + np.exp(-o)), final, h


def recurrence_backward(dy, x, forget, cu, gate=None, state=None, reverse=False, dfinal=None):
    """(dx, dforget, dgate, dstate) of the loss sum(dy * y) + sum(dfinal * final)."""
    dy, x, z = (np.asarray(t, np.float64) for t in (dy, x, forget))
    _, _, h = recurrence(x, z, cu, None, state, reverse)
    o = None if gate is None else np.asarray(gate, np.float64)
    dx, dz, do = (np.full(x.shape, np.nan) for _ in range(3))
    dstate = np.zeros((len(cu) - 1,) + x.shape[1:]) if dfinal is None else np.array(dfinal, np.float64)
    for i, run in enumerate(_runs(cu, reverse)):
        for k in reversed(range(len(run))):
            t = run[k]
            before = h[run[k - 1]] if k else (0 if state is None else np.asarray(state, np.float64)[i])
            direct = dy[t]
            if o is not None:
                sig = 1 / (1 + np.exp(-o[t]))
                do[t] = dy[t] * h[t] * sig * (1 + o[t] * (1 - sig))
                direct = dy[t] * o[t] * sig
            dh = direct + dstate[i]
            f, keep = 1 / (1 + np.exp(-z[t])), 1 / (1 + np.exp(z[t]))
            dx[t] = keep * dh
            dz[t] = dh * (before - x[t]) * f * keep
            dstate[i] = f * dh
    return dx, dz, None if gate is None else do, dstate


def seen_position(pos, g, G, d4=False):
    """Positions [N, axes] as group element g sees them: the last two turned by its inverse."""
    p = np.array(pos, np.float64)
    if p.shape[1] < 2 or G == 1:
        return p
    a = (g % 4) * np.pi / 2 if d4 else 2 * np.pi * g / G
    turn = np.array([[np.cos(a), -np.sin(a)], [np.sin(a), np.cos(a)]])  # R^g on (row, column)
    if d4 and g >= 4:
        turn = turn @ np.diag([1.0, -1.0])
    p[:, -2:] = p[:, -2:] @ np.linalg.inv(turn).T
    return p


def rotary(x, pos, pairs, base=10000.0, d4=False, inverse=False):
    """x [N, H, dc, G] turned by pos [N, axes]."""
    x = np.asarray(x, np.float64)
    y, P, G = x.copy(), sum(pairs), x.shape[3]
    for g in range(G):
        p, j = seen_position(pos, g, G, d4), 0
        for axis, count in enumerate(pairs):
            for i in range(count):
                t = p[:, axis] * base ** (-i / count) * (-1 if inverse else 1)
                c, s = np.cos(t)[:, None], np.sin(t)[:, None]
                a, b = x[:, :, j, g], x[:, :, j + P, g]
                y[:, :, j, g], y[:, :, j + P, g] = a * c - b * s, a * s + b * c
                j += 1
    return y


def _sequences(cu_q, cu_k, len_k):
    for i in range(len(cu_q) - 1):
        lk = cu_k[i + 1] - cu_k[i] if len_k is None else min(len_k[i], cu_k[i + 1] - cu_k[i])
        yield slice(cu_q[i], cu_q[i + 1]), slice(cu_k[i], cu_k[i] + lk), cu_q[i + 1] - cu_q[i], lk


def _softmax(s, see):
    """Rows of s over the allowed places: (p, lse); a row without any is zeros and -inf."""
    p, lse = np.zeros_like(s), np.full(s.shape[0], -np.inf)
    for t in range(s.shape[0]):
        at = see[t]
        if at.any():
            m = s[t, at].max()
            e = np.exp(s[t, at] - m)
            p[t, at] = e / e.sum()
            lse[t] = m + np.log(e.sum())
    return p, lse


def _see(lq, lk, causal):
    return (np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)) if causal else np.ones((lq, lk), bool)


def attention(q, k, v, cu_q, cu_k, causal=False, scale=None, len_k=None):
    """(o, lse) of q [Tq, Hq, D], k and v [Tk, Hkv, D]. Only the keys a token sees enter its sums."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    grp = q.shape[1] // k.shape[1]
    for rq, rk, lq, lk in _sequences(cu_q, cu_k, len_k):
        see = _see(lq, lk, causal)
        for h in range(q.shape[1]):
            with np.errstate(invalid="ignore"):  # values of keys that are not seen may be anything
                s = q[rq, h] @ k[rk, h // grp].T * scale
            p, lse[rq, h] = _softmax(s, see)
            vals = v[rk, h // grp]
            fine = np.isfinite(vals).all(axis=1)
            o[rq, h] = p[:, fine] @ vals[fine]
            for j in np.flatnonzero(~fine):
                for t in np.flatnonzero(see[:, j]):
                    o[rq.start + t, h] += p[t, j] * vals[j]
    return o, lse


def attention_backward(do, q, k, v, cu_q, cu_k, causal=False, scale=None, len_k=None):
    """(dq, dk, dv) of the loss sum(do * o)."""
    do, q, k, v = (np.asarray(t, np.float64) for t in (do, q, k, v))
    scale = q.shape[2] ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    grp = q.shape[1] // k.shape[1]
    for rq, rk, lq, lk in _sequences(cu_q, cu_k, len_k):
        see = _see(lq, lk, causal)
        for h in range(q.shape[1]):
            g = h // grp
            p, _ = _softmax(q[rq, h] @ k[rk, g].T * scale, see)
            dp = do[rq, h] @ v[rk, g].T
            ds = p * (dp - (p * dp).sum(axis=1, keepdims=True)) * scale
            dv[rk, g] += p.T @ do[rq, h]
            dq[rq, h] = ds @ k[rk, g]
            dk[rk, g] += ds.T @ q[rq, h]
    return dq, dk, dv
