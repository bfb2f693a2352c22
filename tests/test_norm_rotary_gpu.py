"""GPU parity of eqlin_rmsnorm, its 8-bit form and backward, and of eqlin_rotary, with the fp64 oracle
(oracle/stage.py) on the same rounded inputs.

Bars (u: the unit roundoff, bf16 2^-8, fp16 2^-11, fp32 2^-24): a stored value is rounded once from fp32 work of relative
error under 1e-6 (sums of squares of up to 2^17 terms): u |ref| + 1e-6 scale, times 1.01, with scale the size of
the terms (for dx: |ds| + rstd (|w| + |xh mean|); rotary: |a| + |b|). dgamma: fp32 sums over N G products,
1e-6 * sqrt(N G) * rms product. e4m3: the scale to 2e-6; q to half a step of its binade around y / scale (1/16
relative or 2^-10 absolute), and the same code as the oracle's except where y / scale is within 1e-5 of a tie.
fp16 also has 2^-25 absolute, half its subnormal step.
"""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def _np(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _near(got, want, scale, dtype, label):
    got = _np(got)
    bar = 1.01 * (U[dtype] * np.abs(want) + 1e-6 * scale) + (2.0 ** -25 if dtype == "f16" else 1e-37)
    worst = float((np.abs(got - want) / bar).max()) if got.size else 0.0
    print(f"[parity] {label}: worst {worst:.3f} of the bar", flush=True)
    assert np.isfinite(got).all() and worst <= 1.0, (label, worst)


def _draw(shape, dtype, dev, gen):
    return torch.randn(shape, generator=gen).to(DT[dtype]).to(dev)


# (N, C, G): one lane, every register form, the element form (odd rows, long rows), many rows
NORM = [(1, 1, 1), (3, 5, 1), (7, 3, 2), (5, 1, 8), (8, 192, 4), (300, 96, 4), (130, 64, 8), (33, 131, 1), (9, 1000, 2),
        (6, 2048, 2), (5, 1500, 8), (3, 2048, 8), (2, 5001, 4), (3000, 16, 4), (2, 16384, 8), (0, 8, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,C,G", NORM)
def test_rmsnorm(N, C, G, dtype, cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(N + C)
    label = f"rmsnorm N={N} C={C} G={G} {dtype}"
    print(f"[case] {label}", flush=True)
    x, r, dy, ds = (_draw((N, C, G), dtype, dev, gen) for _ in range(4))
    gamma = (1 + 0.2 * torch.randn(C, generator=gen)).to(DT[dtype]).to(dev)
    for g, res in ((gamma, r), (None, None), (gamma, None)):
        y, s, rstd = eq.rmsnorm(x, g, residual=res, eps=1e-5)
        q, scale, s2, rstd2 = eq.rmsnorm_quant(x, g, residual=res, eps=1e-5)
        torch.cuda.synchronize()
        assert torch.equal(s, s2) and torch.equal(rstd, rstd2)
        if N == 0:
            continue
        gn, rn = None if g is None else _np(g), None if res is None else _np(res)
        wy, ws, wr = stage.rmsnorm(_np(x), gn, rn, 1e-5)
        assert np.abs(_np(rstd) / wr - 1).max() <= 2e-6
        _near(s, ws, np.abs(ws), dtype, label + " s")
        _near(y, wy, np.abs(wy), dtype, label + " y")
        wq, wscale, _, _ = stage.rmsnorm_quant(_np(x), gn, rn, 1e-5)
        assert np.abs(_np(scale) / wscale - 1).max() <= 2e-6
        t, got = wy / wscale[:, None, None], _np(q.float())
        assert (np.abs(got - t) <= np.maximum(np.abs(t) / 16, 2.0 ** -10) * (1 + 1e-4)).all()
        tie = np.abs(np.abs(t - got) - np.abs(t - wq)) <= 1e-5 * np.abs(t)
        assert ((got == wq) | tie).all(), label
    y, s, rstd = eq.rmsnorm(x, gamma, residual=r)
    for g, d in ((gamma, ds), (None, None)):
        dx, dgamma = eq.rmsnorm_backward(dy, s, g, rstd, ds=d)
        dx2, none = eq.rmsnorm_backward(dy, s, g, rstd, ds=d, with_gamma=False)
        torch.cuda.synchronize()
        assert none is None and torch.equal(dx, dx2)
        if N == 0:
            assert not dgamma.any()
            continue
        gn, dn = None if g is None else _np(g), None if d is None else _np(d)
        wdx, wdg = stage.rmsnorm_backward(_np(dy), _np(s), gn, _np(rstd), dn)
        w = _np(dy) * (1 if g is None else gn[None, :, None])
        xh = _np(s) * _np(rstd)[:, None, None]
        scale = (0 if d is None else np.abs(dn)) + _np(rstd)[:, None, None] * (
            np.abs(w) + np.abs(xh) * np.abs(w * xh).mean(axis=(1, 2))[:, None, None])
        _near(dx, wdx, scale, dtype, label + " dx")
        bar = 1e-6 * np.sqrt(N * G) * np.sqrt(((_np(dy) * xh) ** 2).mean(axis=(0, 2))) + 1e-6 * np.abs(wdg) + 1e-6
        assert (np.abs(_np(dgamma) - wdg) <= bar).all(), (label, np.abs(_np(dgamma) - wdg).max())


def test_rmsnorm_rows_that_are_special(cuda_device):
    """Zero rows, infinities, NaN and the type's largest values stay in their rows."""
    dev = cuda_device
    x = torch.randn((6, 40, 4), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(dev)
    x[1] = 0
    x[2, 3, 1] = float("inf")
    x[3, 5, 2] = float("nan")
    x[4] = 3e38
    y, s, rstd = eq.rmsnorm(x, eps=0.0)
    q, scale, _, _ = eq.rmsnorm_quant(x, eps=1e-6)
    torch.cuda.synchronize()
    want, _, _ = stage.rmsnorm(_np(x[[0, 5]]), eps=0.0)
    _near(y[[0, 5]], want, np.abs(want), "bf16", "special rows")
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all())  # 0 * inf with eps = 0; NaN
    assert float(scale[1]) == 1.0 and not q[1].float().any()
    assert bool(q[3].float().isnan().all()) and bool(y[2, 3, 1].isnan()) and not y[2, 0].any()
    assert bool(torch.isinf(rstd[1])) and float(rstd[4]) == 0.0 and not y[4].any()  # 1/sqrt of an infinite sum


def test_rmsnorm_group_shift_and_refusals(cuda_device):
    dev = cuda_device
    x = torch.randn((9, 24, 8), generator=torch.Generator().manual_seed(1)).to(dev)
    gamma = torch.rand(24, generator=torch.Generator().manual_seed(2)).to(dev)
    y, _, _ = eq.rmsnorm(x, gamma)
    y2, _, _ = eq.rmsnorm(x.roll(3, 2).contiguous(), gamma)
    assert float((y2 - y.roll(3, 2)).abs().max()) <= 1e-6 * float(y.abs().max())
    rstd = torch.ones(9, device=dev)
    for kind, call in [
        (ValueError, lambda: eq.rmsnorm(x[0])), (ValueError, lambda: eq.rmsnorm(x, gamma[:5])),
        (ValueError, lambda: eq.rmsnorm(x, gamma.half())), (ValueError, lambda: eq.rmsnorm(x, residual=x[:8])),
        (ValueError, lambda: eq.rmsnorm(x.transpose(0, 1))), (TypeError, lambda: eq.rmsnorm(x.cpu())),
        (TypeError, lambda: eq.rmsnorm(x.double())), (eq.EqlinError, lambda: eq.rmsnorm(x, eps=-1.0)),
        (eq.EqlinError, lambda: eq.rmsnorm(x, eps=float("nan"))), (eq.EqlinError, lambda: eq.rmsnorm(x, y=x)),
        (eq.EqlinError, lambda: eq.rmsnorm(x[:, :, :3].contiguous())),
        (ValueError, lambda: eq.rmsnorm_backward(x, x, gamma, rstd[:3])),
        (ValueError, lambda: eq.rmsnorm_backward(x[:3], x, gamma, rstd)),
    ]:
        with pytest.raises(kind):
            call()


# (N, H, dc, G, pairs, group)
ROTARY = [(1, 1, 2, 1, (1,), "cyclic"), (5, 3, 128, 1, (16, 24, 24), "cyclic"), (70, 8, 16, 8, (4, 4), "cyclic"),
          (33, 5, 16, 4, (3, 3), "cyclic"), (40, 2, 8, 8, (2, 2), "d4"), (17, 3, 7, 8, (1, 2), "d4"), (12, 2, 32, 2, (16,), "cyclic"),
          (20, 4, 24, 4, (2, 0, 4), "cyclic"), (9, 2, 21, 1, (2, 3, 2, 3), "cyclic"), (300, 12, 64, 1, (32,), "cyclic")]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", ROTARY, ids=[f"r{i}" for i in range(len(ROTARY))])
def test_rotary(case, dtype, cuda_device):
    N, H, dc, G, pairs, group = case
    dev, gen = cuda_device, torch.Generator().manual_seed(N)
    label = f"rotary N={N} H={H} dc={dc} G={G} pairs={pairs} {group} {dtype}"
    print(f"[case] {label}", flush=True)
    pos = torch.randint(-300, 4000, (N, len(pairs)), generator=gen).to(torch.int32)
    pos[0] = 1 << 22
    wide = _draw((N, H + 2, dc, G), dtype, dev, gen)
    for x, first in ((wide[:, :H].contiguous(), 0), (wide[:, 1:H + 1], 1)):
        for inverse in (False, True):
            before = x.clone()
            y = eq.rotary(x, pos.to(dev), pairs, group=group, inverse=inverse)
            z = wide.clone()[:, first:first + H]
            eq.rotary(z, pos.to(dev), pairs, group=group, inverse=inverse, out=z)
            torch.cuda.synchronize()
            assert torch.equal(x, before) and torch.equal(y, z)
            want = stage.rotary(_np(x), pos.numpy(), pairs, d4=group == "d4", inverse=inverse)
            P = sum(pairs)
            pair = np.abs(_np(x[:, :, :P])) + np.abs(_np(x[:, :, P:2 * P]))
            scale = np.concatenate([pair, pair, np.zeros_like(_np(x[:, :, 2 * P:]))], 2)
            # half types: sine and cosine to 2e-6 absolute
            _near(y, want, scale * (1 if dtype == "f32" else 3), dtype, label)


def test_rotary_refusals(cuda_device):
    x = torch.zeros((4, 2, 8, 4), device=cuda_device)
    pos = torch.zeros((4, 2), dtype=torch.int32, device=cuda_device)
    for kind, call in [
        (ValueError, lambda: eq.rotary(x, pos, (2,))), (ValueError, lambda: eq.rotary(x, pos.long(), (2, 2))),
        (ValueError, lambda: eq.rotary(x, pos[:3], (2, 2))), (ValueError, lambda: eq.rotary(x, pos, (2, 2), group="so2")),
        (ValueError, lambda: eq.rotary(x.transpose(2, 3), pos, (2, 2))), (TypeError, lambda: eq.rotary(x.double(), pos, (2, 2))),
        (eq.EqlinError, lambda: eq.rotary(x, pos, (3, 2))), (eq.EqlinError, lambda: eq.rotary(x, pos, (0, 0))),
        (eq.EqlinError, lambda: eq.rotary(x, pos, (-1, 2))), (eq.EqlinError, lambda: eq.rotary(x, pos, (2, 2), base=0.0)),
        (eq.EqlinError, lambda: eq.rotary(x, pos, (2, 2), group="d4")),
        (eq.EqlinError, lambda: eq.rotary(x[:2], pos[:2], (2, 2), out=x[1:3])),
        (eq.EqlinError, lambda: eq.rotary(x, pos, (2, 2), out=x[:1].clone().expand(4, 2, 8, 4))),
    ]:
        with pytest.raises(kind):
            call()
    e = eq.rotary(x[:0], pos[:0], (2, 2))
    assert e.shape == (0, 2, 8, 4)
