"""The operators of a transformer stage run together (examples/eq_stage.py): equivariance of the whole stage, its
attention half's gradients against differences, and graph replays of the operators."""
import os
import sys

import pytest
import torch

import fourier_domain_linear_amd as eq

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from eq_stage import Stage, packed_images  # noqa: E402

pytestmark = pytest.mark.gpu


def _x(N, C, G, dtype, dev, seed=3):
    return torch.randn((N, C, G), generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev)


@pytest.mark.parametrize("dtype,bar", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)], ids=["f32", "bf16"])
def test_stage_commutes_with_a_quarter_turn(dtype, bar, cuda_device):
    """Turned positions and a shifted group axis give the shifted output. Bars: the layers' own parity bars (relative
    Frobenius 1e-5 and 1e-2) twice, for the two sides."""
    stage = Stage(32, 4, 4, dtype, cuda_device)
    pos, cu = packed_images([(7, 9), (5, 4), (1, 1)], cuda_device)
    x = _x(pos.shape[0], 32, 4, dtype, cuda_device)
    turned = torch.stack([-pos[:, 1], pos[:, 0]], 1).contiguous()
    y, s, _ = stage.forward(x, pos, cu)
    y2, s2, _ = stage.forward(x.roll(1, 2).contiguous(), turned, cu)
    for a, b in ((y, y2), (s, s2)):
        a, b = a.double().roll(1, 2), b.double()
        assert float((a - b).norm() / a.norm()) <= bar
    if dtype != torch.float32:
        return
    y3, _, _ = stage.forward(x.roll(1, 2).contiguous(), pos, cu)  # the positions not turned: another function
    assert float((y3.double() - y.double().roll(1, 2)).norm() / y.double().norm()) > 10 * bar


def test_stage_gradients_against_differences(cuda_device):
    """d/dt of sum(dy y2 + ds s2) along random directions of x and of the weights, central differences of the fp32
    forward. Bar: the difference quotient's own rounding, about 2^-24 |loss terms| / h with h = 1e-2, and its h^2
    term: 1e-3 of the size of the terms."""
    dev = cuda_device
    stage = Stage(16, 2, 4, torch.float32, dev)
    pos, cu = packed_images([(4, 5), (3, 3)], dev)
    N = pos.shape[0]
    x = _x(N, 16, 4, torch.float32, dev)
    dy, ds = _x(N, 16, 4, torch.float32, dev, 4), _x(N, 16, 4, torch.float32, dev, 5)

    def loss(x, W=None):
        kept_layers = dict(stage.layer)
        for n, w in (W or {}).items():
            stage.layer[n] = eq.prepare_weights(w, backward=True)
        _, _, kept = stage.forward(x, pos, cu)
        stage.layer.update(kept_layers)
        return float((dy.double() * kept["y2"].double() + ds.double() * kept["s2"].double()).sum())

    _, _, kept = stage.forward(x, pos, cu)
    dx, grads = stage.attention_backward(dy, ds, pos, cu, kept)
    h = 1e-2
    for seed in range(3):
        d = _x(N, 16, 4, torch.float32, dev, 10 + seed)
        want = (loss(x + h * d) - loss(x - h * d)) / (2 * h)
        got = float((dx.double() * d.double()).sum())
        assert abs(got - want) <= 1e-3 * float((dx.double() * d.double()).abs().sum()), (seed, got, want)
        for n in ("qkv", "out"):
            w = stage.W[n]
            d = _x(*w.shape, torch.float32, dev, 20 + seed) * w.shape[1] ** -0.5
            want = (loss(x, {n: (w + h * d).contiguous()}) - loss(x, {n: (w - h * d).contiguous()})) / (2 * h)
            got = float((grads[n].double() * d.double()).sum())
            assert abs(got - want) <= 1e-3 * float((grads[n].double() * d.double()).abs().sum()), (n, seed, got, want)


def test_operators_in_a_graph(cuda_device):
    """Captured and replayed four times with eager work between: the same bits as the eager calls."""
    dev = cuda_device
    gen = torch.Generator().manual_seed(0)
    x, r = (torch.randn((130, 96, 4), generator=gen).bfloat16().to(dev) for _ in range(2))
    gamma = torch.rand(96, generator=gen).bfloat16().to(dev)
    q = torch.randn((130, 6, 64), generator=gen).bfloat16().to(dev)
    step = torch.randn((2, 6, 64), generator=gen).bfloat16().to(dev)
    kv = torch.randn((2, 2000, 2, 64), generator=gen).bfloat16().to(dev)
    pos = torch.randint(0, 50, (130, 3), generator=gen).to(torch.int32).to(dev)
    cu = torch.tensor([0, 50, 130], dtype=torch.int32, device=dev)
    cu1, cuk = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev), torch.tensor([0, 1500, 2000], dtype=torch.int32, device=dev)

    def run():
        y, s, rstd = eq.rmsnorm(x, gamma, residual=r)
        c, scale, _, _ = eq.rmsnorm_quant(x, gamma, residual=r)
        dx, dg = eq.rmsnorm_backward(y, s, gamma, rstd, ds=x)
        t = eq.rotary(q, pos, (8, 12, 12))
        o, lse = eq.attention(t, t, q, cu, cu, causal=True)
        g = eq.attention_backward(q, t, t, q, o, lse, cu, cu, causal=True)
        o1, lse1 = eq.attention(step, kv[0], kv[1], cu1, cuk, causal=True)
        return [y, s, rstd, c.view(torch.uint8), scale, dx, dg, t, o, lse, *g, o1, lse1]

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        again = run()
        torch.cuda.synchronize()
        for a, b in zip(again, want):
            assert torch.equal(a, b)
