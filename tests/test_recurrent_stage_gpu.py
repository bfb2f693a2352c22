"""The operators of a recurrent stage run together (examples/eq_recurrent_stage.py): against the fp64 oracle, under a shift of the
group axis, in pieces with the states handed on, its mixing half's gradients against differences, and in a captured graph."""
import os
import sys

import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
import oracle
from oracle import stage as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from eq_recurrent_stage import RecurrentStage, main  # noqa: E402

pytestmark = pytest.mark.gpu


def _x(N, C, G, dtype, dev, seed=3):
    return torch.randn((N, C, G), generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev)


def _cu(lens, dev):
    return torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)


def _oracle(stage, x, edges, state, reverse):
    n = lambda t: t.detach().to("cpu", torch.float64).numpy()  # noqa: E731
    cpu = lambda t: t.detach().cpu()  # noqa: E731
    lin = lambda name, t: np.asarray(oracle.forward(torch.from_numpy(t).float(), cpu(stage.W[name]).float(), cpu(stage.b[name]).float()))  # noqa: E731
    C, g, b = stage.C, [n(t) for t in stage.gamma], [n(t) for t in stage.beta]
    x = n(x)
    mix = lin("mix", ref.layernorm(x, g[0], b[0])[0])
    h, final, _ = ref.recurrence(mix[:, :C], mix[:, C:2 * C], edges, mix[:, 2 * C:], n(state), reverse)
    y2, s2, _, _ = ref.layernorm(lin("out", h), g[1], b[1], x)
    m = lin("down", np.asarray(oracle.gelu(lin("up", y2))))
    return ref.layernorm(m, g[2], b[2], s2)[:2] + (final,)


@pytest.mark.parametrize("reverse", [False, True])
def test_stage_against_the_oracle(reverse, cuda_device):
    """fp32. Bar: the layers' own relative Frobenius bar of 1e-5, four layers one after the other, and the fp32 rounding of
    what the oracle's layers are fed."""
    dev, lens = cuda_device, [70, 1, 300, 9]
    stage = RecurrentStage(16, 4, torch.float32, dev, reverse=reverse)
    x, h0 = _x(sum(lens), 16, 4, torch.float32, dev), _x(4, 16, 4, torch.float32, dev, 4)
    for longest in (None, 300):
        got = stage.forward(x, _cu(lens, dev), h0, longest=longest)[:3]
        torch.cuda.synchronize()
        want = _oracle(stage, x, [0, 70, 71, 371, 380], h0, reverse)
        for a, b in zip(got, want):
            a = a.double().cpu().numpy()
            assert np.linalg.norm(a - b) <= 4e-5 * np.linalg.norm(b)


@pytest.mark.parametrize("dtype,bar", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)], ids=["f32", "bf16"])
def test_stage_commutes_with_a_shift_of_the_group_axis(dtype, bar, cuda_device):
    """Bars: the layers' own parity bars (relative Frobenius 1e-5 and 1e-2) twice, for the two sides."""
    dev, lens = cuda_device, [130, 40]
    stage = RecurrentStage(32, 4, dtype, dev)
    x, h0 = _x(170, 32, 4, dtype, dev), _x(2, 32, 4, torch.float32, dev, 4)
    roll = lambda t: t.roll(1, 2).contiguous()  # noqa: E731
    a = stage.forward(x, _cu(lens, dev), h0)[:3]
    b = stage.forward(roll(x), _cu(lens, dev), roll(h0))[:3]
    for p, q in zip(a, b):
        p, q = p.double().roll(1, 2), q.double()
        assert float((p - q).norm() / p.norm()) <= bar


def test_prompts_then_tokens_equal_whole_sequences(cuda_device):
    """Prompts of different lengths in one call, then the streams' tokens one at a time with the states handed on. fp32; the same
    sums in another order: 2e-5 of the size."""
    dev, streams, prompt, more = cuda_device, 3, [5, 80, 33], 4
    stage = RecurrentStage(16, 8, torch.float32, dev)
    lens = [n + more for n in prompt]
    x = _x(sum(lens), 16, 8, torch.float32, dev)
    whole, _, final, _ = stage.forward(x, _cu(lens, dev))
    starts = [0, lens[0], lens[0] + lens[1]]
    rows = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, prompt)]).to(dev)
    y, _, state, _ = stage.forward(x[rows], _cu(prompt, dev))
    assert float((y - whole[rows]).abs().max()) <= 2e-5 * float(whole.abs().max())
    one = torch.arange(streams + 1, device=dev, dtype=torch.int32)
    for k in range(more):
        rows = torch.tensor([s + n + k for s, n in zip(starts, prompt)], device=dev)
        y, _, state, _ = stage.forward(x[rows], one, state, longest=1)
        assert float((y - whole[rows]).abs().max()) <= 2e-5 * float(whole.abs().max())
    assert float((state - final).abs().max()) <= 2e-5 * float(final.abs().max())


def test_stage_gradients_against_differences(cuda_device):
    """d/dt of sum(dy y2 + ds s2 + dfinal final) along random directions of x, the initial states, the weights and the norms'
    parameters, central differences of the fp32 forward. Bar: the difference quotient's own rounding, about 2^-24 |loss
    terms| / h with h = 1e-2, and its h^2 term: 1e-3 of the size of the terms."""
    dev, lens = cuda_device, [70, 0, 5]
    stage = RecurrentStage(16, 4, torch.float32, dev)
    cu, N = _cu(lens, dev), sum(lens)
    x, h0 = _x(N, 16, 4, torch.float32, dev), _x(3, 16, 4, torch.float32, dev, 6)
    dy, ds, dfinal = _x(N, 16, 4, torch.float32, dev, 4), _x(N, 16, 4, torch.float32, dev, 5), _x(3, 16, 4, torch.float32, dev, 7)

    def loss(x=x, h0=h0):
        _, _, final, kept = stage.forward(x, cu, h0)
        return float((dy.double() * kept["y2"].double() + ds.double() * kept["s2"].double()).sum() + (dfinal.double() * final.double()).sum())

    _, _, _, kept = stage.forward(x, cu, h0, training=True)
    dx, dh0, grads = stage.mix_backward(dy, ds, cu, kept, dfinal)
    h = 1e-2

    def near(grad, d, up, down, label):
        terms = grad.double() * d.double()
        assert abs(float(terms.sum()) - (up - down) / (2 * h)) <= 1e-3 * float(terms.abs().sum()), label

    for seed in range(2):
        d = _x(N, 16, 4, torch.float32, dev, 10 + seed)
        near(dx, d, loss(x=x + h * d), loss(x=x - h * d), ("x", seed))
        d = _x(3, 16, 4, torch.float32, dev, 20 + seed)
        near(dh0, d, loss(h0=h0 + h * d), loss(h0=h0 - h * d), ("state", seed))
        for n in ("mix", "out"):
            w, layer = stage.W[n], stage.layer[n]
            d = _x(*w.shape, torch.float32, dev, 30 + seed) * w.shape[1] ** -0.5
            sides = []
            for sign in (1, -1):
                stage.layer[n] = eq.prepare_weights((w + sign * h * d).contiguous(), backward=True)
                sides.append(loss())
            stage.layer[n] = layer
            near(grads[n], d, *sides, (n, seed))
        for name, params in (("gamma", stage.gamma), ("beta", stage.beta)):
            for k in range(2):
                p = params[k]
                d = torch.randn(16, generator=torch.Generator().manual_seed(40 + seed)).to(dev)
                sides = []
                for sign in (1, -1):
                    params[k] = p + sign * h * d
                    sides.append(loss())
                params[k] = p
                near(grads[f"{name}{k + 1}"], d, *sides, (name, k, seed))


def test_steps_in_a_graph_update_their_states(cuda_device):
    """A captured step whose states are updated in place: each replay is the next token of every stream."""
    dev, B = cuda_device, 40
    gen = torch.Generator().manual_seed(1)
    mix, state = torch.zeros((B, 48, 4), device=dev).bfloat16(), torch.zeros((B, 16, 4), device=dev)
    gamma, beta = torch.rand(16, generator=gen).bfloat16().to(dev), torch.rand(16, generator=gen).bfloat16().to(dev)
    cu = torch.arange(B + 1, device=dev, dtype=torch.int32)

    def step(state):
        y, _, _ = eq.recurrence(mix[:, :16], mix[:, 16:32], cu, gate=mix[:, 32:], state=state, final=state, longest=1)
        return eq.layernorm(y, gamma, beta)[0]

    step(state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(state)
    state.zero_()
    eager = torch.zeros_like(state)
    for _ in range(4):
        mix.copy_(torch.randn(mix.shape, generator=gen).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, eager) and bool(state.any())


def test_example_runs(cuda_device, capsys):
    main()
    assert "streams" in capsys.readouterr().out
