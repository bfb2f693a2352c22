"""GPU parity of eqlin_layernorm and its backward with the fp64 oracle (oracle/stage.py) on the same rounded inputs.

Bars (u: the unit roundoff, bf16 2^-8, fp16 2^-11, fp32 2^-24): a stored value is rounded once from fp32 work. There every value
of the centred row carries the rounding of s and of the mean (sums in trees and chains of at most 64 additions a lane's
part: under 1e-6 of the mean magnitude), and mean square and rstd the relative error of those, so
y's scale is |gamma| (|xh| + R (1 + |xh|)) + |beta| with R = rstd (|s| + mean |s|), the bar u |y| + 1e-6 scale, times 1.01.
rstd: 2e-6 (1 + max of R^2 over the row's rms...) is covered by the same R. dx: X = |xh| + rstd (|s| + |mean|) is xh with the
rounding of s - mean; scale |ds| + rstd (|w| + mean |w| + X mean(|w| X)). dgamma, dbeta: fp32 sums, 1e-6 of the sum of
|dy| X and of |dy|. fp16 also has 2^-25 absolute, half its subnormal step.
"""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage
from test_norm_rotary_gpu import DT, _draw, _near, _np

pytestmark = pytest.mark.gpu

# (N, C, G): one lane, each register form at each load width (16 bytes, 4 bytes, one element), the long rows, many rows
SHAPES = [(1, 1, 1), (3, 5, 1), (7, 3, 2), (5, 1, 8), (8, 192, 4), (300, 96, 4), (130, 64, 8), (33, 131, 1), (2500, 181, 1), (9, 1000, 2),
          (6, 2048, 2), (5, 1500, 8), (3, 2048, 8), (4, 97, 2), (11, 333, 2), (6, 1025, 2), (5, 1501, 1), (3, 2303, 1), (2, 5001, 4), (2, 4097, 2),
          (3000, 16, 4), (2, 16384, 8), (3, 9000, 1), (0, 8, 4)]


def _check(x, r, gamma, beta, dy, ds, dtype, label):
    """Forward and gradients of one call against the oracle."""
    n = lambda t: None if t is None else _np(t)  # noqa: E731
    y, s, mean, rstd = eq.layernorm(x, gamma, beta, residual=r)
    torch.cuda.synchronize()
    wy, ws, wm, wr = stage.layernorm(_np(x), n(gamma), n(beta), n(r))
    _near(s, ws, np.abs(ws), dtype, label + " s")
    R = wr[:, None, None] * (np.abs(ws) + np.abs(ws).mean(axis=(1, 2))[:, None, None])
    g = np.ones(ws.shape[1]) if gamma is None else _np(gamma)
    b = np.zeros(ws.shape[1]) if beta is None else _np(beta)
    xh = (ws - wm[:, None, None]) * wr[:, None, None]
    scale = np.abs(g)[None, :, None] * (np.abs(xh) + R * (1 + np.abs(xh))) + np.abs(b)[None, :, None]
    _near(y, wy, scale, dtype, label + " y")
    assert (np.abs(_np(mean) - wm) <= 1e-6 * np.abs(ws).mean(axis=(1, 2)) + 1e-37).all(), label
    # the squares' mean carries twice the centred values' error
    worst = (R * np.abs(xh)).mean(axis=(1, 2))
    assert (np.abs(_np(rstd) / wr - 1) <= 2e-6 * (1 + worst)).all(), (label, np.abs(_np(rstd) / wr - 1).max())

    dx, dgamma, dbeta = eq.layernorm_backward(dy, s, gamma, mean, rstd, ds=ds)
    dx2, no1, no2 = eq.layernorm_backward(dy, s, gamma, mean, rstd, ds=ds, with_params=False)
    torch.cuda.synchronize()
    assert no1 is None and no2 is None and torch.equal(dx, dx2)
    s64, m64, r64, d64 = _np(s), _np(mean), _np(rstd), _np(dy)
    wdx, wdg, wdb = stage.layernorm_backward(d64, s64, n(gamma), m64, r64, n(ds))
    w = np.abs(d64 * g[None, :, None])
    X = r64[:, None, None] * (np.abs(s64 - m64[:, None, None]) + np.abs(s64) + np.abs(m64)[:, None, None])
    along = lambda t: t.mean(axis=(1, 2))[:, None, None]  # noqa: E731
    scale = (0 if ds is None else np.abs(_np(ds))) + r64[:, None, None] * (w + along(w) + X * along(w * X))
    _near(dx, wdx, scale, dtype, label + " dx")
    assert (np.abs(_np(dgamma) - wdg) <= 1e-6 * (np.abs(d64) * X).sum(axis=(0, 2)) + 1e-30).all(), (label, "dgamma")
    assert (np.abs(_np(dbeta) - wdb) <= 1e-6 * np.abs(d64).sum(axis=(0, 2)) + 1e-30).all(), (label, "dbeta")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,C,G", SHAPES)
def test_layernorm(N, C, G, dtype, cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(N + C)
    label = f"layernorm N={N} C={C} G={G} {dtype}"
    print(f"[case] {label}", flush=True)
    x, r, dy, ds = (_draw((N, C, G), dtype, dev, gen) for _ in range(4))
    gamma, beta = ((k + 0.2 * torch.randn(C, generator=gen)).to(DT[dtype]).to(dev) for k in (1, 0))
    if N == 0:
        y, s, mean, rstd = eq.layernorm(x, gamma, beta, residual=r)
        _, dgamma, dbeta = eq.layernorm_backward(dy, s, gamma, mean, rstd)
        torch.cuda.synchronize()
        assert y.shape == x.shape and not dgamma.any() and not dbeta.any()
        return
    _check(x, r, gamma, beta, dy, ds, dtype, label)
    _check(x, None, None, None, dy, None, dtype, label + " bare")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 67])
def test_a_common_part_many_times_the_spread(C, dtype, cuda_device):
    """The variance is taken about the mean: rows of 300 +- 1 keep their bits."""
    dev, gen = cuda_device, torch.Generator().manual_seed(C)
    x = (300 + 2 * torch.randn((40, C, 4), generator=gen)).to(DT[dtype]).to(dev)
    dy = _draw(x.shape, dtype, dev, gen)
    _check(x, None, None, None, dy, None, dtype, f"common part C={C} {dtype}")


def test_rows_that_are_special(cuda_device):
    """Constant rows, infinities and NaN stay in their rows, in both directions."""
    dev, gen = cuda_device, torch.Generator().manual_seed(0)
    x = torch.randn((6, 40, 4), generator=gen).to(torch.bfloat16).to(dev)
    x[1] = 3
    x[2, 3, 1] = float("inf")
    x[3, 5, 2] = float("nan")
    beta = torch.randn(40, generator=gen).to(torch.bfloat16).to(dev)
    y, s, mean, rstd = eq.layernorm(x, None, beta)
    dy = torch.randn(x.shape, generator=gen).to(torch.bfloat16).to(dev)
    dx, _, _ = eq.layernorm_backward(dy, s, None, mean, rstd)
    torch.cuda.synchronize()
    want = stage.layernorm(_np(x[[0, 4, 5]]), None, _np(beta))
    _near(y[[0, 4, 5]], want[0], 4 * (np.abs(want[0]) + 1), "bf16", "fine rows")
    assert torch.equal(y[1], beta[:, None].expand(40, 4)) and float(mean[1]) == 3.0
    assert bool(y[2].isnan().all()) and bool(y[3].isnan().all())
    assert bool(dx[[0, 1, 4, 5]].isfinite().all()) and bool(dx[2].isnan().all()) and bool(dx[3].isnan().all())
    y, _, _, rstd = eq.layernorm(x[1:2].contiguous(), eps=0.0)  # 0 times 1 / 0
    torch.cuda.synchronize()
    assert bool(torch.isinf(rstd).all()) and bool(y.isnan().all())


def test_gradients_by_differences(cuda_device):
    """dx, dgamma and dbeta against central differences of the kernel's own forward (fp32, h = 2^-6: third-order terms of size
    h^2, and rounding of 2^-24 |sum| / h)."""
    dev, gen = cuda_device, torch.Generator().manual_seed(3)
    x, dy = (torch.randn((3, 6, 4), generator=gen).to(dev) for _ in range(2))
    gamma, beta = (torch.randn(6, generator=gen).to(dev) for _ in range(2))
    loss = lambda a, g, b: float((eq.layernorm(a, g, b)[0].double() * dy.double()).sum())  # noqa: E731
    _, s, mean, rstd = eq.layernorm(x, gamma, beta)
    grads = eq.layernorm_backward(dy, s, gamma, mean, rstd)
    h = 2.0 ** -6
    for k, t in enumerate((x, gamma, beta)):
        args = [x, gamma, beta]
        for i in range(0, t.numel(), 5):
            step = torch.zeros_like(t).view(-1)
            step[i] = h
            up, down = (loss(*[a if j != k else t + sign * step.view_as(t) for j, a in enumerate(args)]) for sign in (1, -1))
            want = (up - down) / (2 * h)
            assert abs(float(grads[k].view(-1)[i]) - want) <= 4e-3, (k, i)


def test_group_shift_streams_graphs_and_refusals(cuda_device):
    dev, gen = cuda_device, torch.Generator().manual_seed(1)
    x, r, dy = (torch.randn((9, 24, 8), generator=gen).to(dev) for _ in range(3))
    gamma, beta = torch.rand(24, generator=gen).to(dev), torch.rand(24, generator=gen).to(dev)
    y, s, mean, rstd = eq.layernorm(x, gamma, beta, residual=r)
    y2, _, _, _ = eq.layernorm(x.roll(3, 2).contiguous(), gamma, beta, residual=r.roll(3, 2).contiguous())
    assert float((y2 - y.roll(3, 2)).abs().max()) <= 1e-5 * float(y.abs().max())
    dx, dg, db = eq.layernorm_backward(dy, s, gamma, mean, rstd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = (*eq.layernorm(x, gamma, beta, residual=r), *eq.layernorm_backward(dy, s, gamma, mean, rstd))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gy, gs, gm, gr = eq.layernorm(x, gamma, beta, residual=r)
            gdx, gdg, gdb = eq.layernorm_backward(dy, gs, gamma, gm, gr)
    side.synchronize()
    for a, b in zip(again, (y, s, mean, rstd, dx, dg, db)):
        assert torch.equal(a, b)
    for k in range(4):  # each replay against the eager result for the inputs of that time
        x.copy_(torch.randn((9, 24, 8), generator=gen))
        want = eq.layernorm(x, gamma, beta, residual=r)
        want = (*want, *eq.layernorm_backward(dy, want[1], gamma, want[2], want[3]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((gy, gs, gm, gr, gdx, gdg, gdb), want):
            assert torch.equal(a, b), k
    for kind, call in [
        (ValueError, lambda: eq.layernorm(x[0])), (ValueError, lambda: eq.layernorm(x, gamma[:5])),
        (ValueError, lambda: eq.layernorm(x, gamma, beta[:5])), (ValueError, lambda: eq.layernorm(x, gamma, beta.half())),
        (ValueError, lambda: eq.layernorm(x, residual=x[:8])), (ValueError, lambda: eq.layernorm(x.transpose(0, 1))),
        (TypeError, lambda: eq.layernorm(x.cpu())), (TypeError, lambda: eq.layernorm(x.double())),
        (eq.EqlinError, lambda: eq.layernorm(x, eps=-1.0)), (eq.EqlinError, lambda: eq.layernorm(x, eps=float("nan"))),
        (eq.EqlinError, lambda: eq.layernorm(x, y=x)), (eq.EqlinError, lambda: eq.layernorm(x[:, :, :3].contiguous())),
        (ValueError, lambda: eq.layernorm_backward(x, x, gamma, rstd[:3], rstd)),
        (ValueError, lambda: eq.layernorm_backward(x, x, gamma, rstd, rstd.half())),
        (ValueError, lambda: eq.layernorm_backward(x[:3], x, gamma, rstd, rstd)),
    ]:
        with pytest.raises(kind):
            call()
