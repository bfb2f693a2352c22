"""GPU parity of eqlin_recurrence and its backward with the fp64 oracle (oracle/stage.py) on the same rounded inputs.

Bars (u: the unit roundoff, bf16 2^-8, fp16 2^-11, fp32 2^-24). f and 1 - f carry a relative error of some units of fp32 (half
types: of the exponent's product with log2 e besides, |z| 2^-24 for |z| up to 12), every step adds two roundings, and a step's
error fades with f. So the state's error is at most eps times a sum of magnitudes that itself runs through the recurrence,
M_t = f M_{t-1} + f |h_{t-1}| + (1 - f) |x_t| with M = |state| in front, eps = 1e-6 (16 units; fp32) or 3e-6. The way back
likewise: dh_t = d_t + f dh_{t+1} is off by eps times D_t = |d_t| + |dh_t| + f_{t+1} (D_{t+1} + |dh_{t+1}|), d = dy silu(gate). Results add the relative errors of their factors (2e-6; half types 4e-6) and one
rounding u |y|; fp16 also 2^-25 absolute, half its subnormal step.
"""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage
from test_norm_rotary_gpu import DT, U, _np

pytestmark = pytest.mark.gpu

LENS = {"one": [1], "steps": [1] * 9, "empties": [0, 1, 0, 0, 17, 0], "edges": [16, 128, 129, 127, 1, 256, 257, 15], "long": [1500, 0, 700, 3]}
WIDTHS = [(1, 1), (3, 1), (65, 1), (16, 8), (33, 2), (97, 4)]


def _inputs(lens, C, G, dtype, dev, seed, lead=0, tail=0, gated=True):
    """Parts of one layer's output, forget gates from half a token's memory to hundreds; rows in front and behind belong to none."""
    gen = torch.Generator().manual_seed(seed)
    T, B, parts = sum(lens) + lead + tail, len(lens), 3 if gated else 2
    p = torch.randn((T, parts * C, G), generator=gen)
    p[:, C:2 * C] += torch.linspace(-1, 6, C)[None, :, None]
    p = p.to(DT[dtype]).to(dev)
    cu = (torch.tensor([0] + lens).cumsum(0) + lead).to(torch.int32)
    rand = lambda *shape: torch.randn(shape, generator=gen).to(dev)  # noqa: E731
    return {"x": p[:, :C], "forget": p[:, C:2 * C], "gate": p[:, 2 * C:] if gated else None, "cu": cu.to(dev), "edges": cu.tolist(),
            "state": rand(B, C, G), "dy": rand(T, C, G).to(DT[dtype]), "dfinal": rand(B, C, G), "parts": p}


def _magnitudes(i, reverse, with_state, with_dfinal, h, wdx):
    """(M of the state after each token, after the last one, in front of each; M of dh at each token, of dstate)."""
    x, z = np.abs(_np(i["x"])), _np(i["forget"])
    f, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    direct = np.abs(_np(i["dy"]))
    if i["gate"] is not None:
        o = _np(i["gate"])
        direct = direct * np.abs(o) / (1 + np.exp(-o))
    M, before, D = (np.zeros(x.shape) for _ in range(3))
    dh = np.abs(wdx) / rest
    start = np.abs(_np(i["state"])) if with_state else np.zeros(_np(i["state"]).shape)
    last, dstate = start.copy(), (np.abs(_np(i["dfinal"])) if with_dfinal else np.zeros(start.shape))
    for k, run in enumerate(stage._runs(i["edges"], reverse)):
        prev = start[k]
        for t in run:
            before[t] = last[k]
            last[k] = f[t] * last[k] + f[t] * prev + rest[t] * x[t]
            M[t], prev = last[k], np.abs(h[t])
        for t in run[::-1]:
            D[t] = direct[t] + dh[t] + dstate[k]
            dstate[k] = f[t] * (D[t] + dh[t])
    return M, last, before, D, dstate


def _near(got, want, bar, label):
    got = _np(got)
    bad = ~np.isfinite(got) | (np.abs(got - want) > bar)
    worst = float(np.nanmax(np.abs(got - want) / bar)) if got.size else 0.0
    print(f"[parity] {label}: worst {worst:.3f} of the bar", flush=True)
    assert not bad.any(), (label, worst, np.argwhere(bad)[:4])


def _check(i, dtype, reverse, longest, label, with_state=True, with_dfinal=True):
    gate, cu, edges = i["gate"], i["cu"], i["edges"]
    state = i["state"] if with_state else None
    dfinal = i["dfinal"] if with_dfinal else None
    out = torch.full(i["x"].shape, 7.0, dtype=DT[dtype], device=cu.device)
    y, final, marks = eq.recurrence(i["x"], i["forget"], cu, gate=gate, state=state, reverse=reverse, longest=longest, with_marks=True, out=out)
    y2, final2, none = eq.recurrence(i["x"], i["forget"], cu, gate=gate, state=state, reverse=reverse, longest=longest)
    grad = torch.full_like(i["parts"], 7.0)
    C = i["x"].shape[1]
    parts = {"dx": grad[:, :C], "dforget": grad[:, C:2 * C], "dgate": None if gate is None else grad[:, 2 * C:]}
    dx, dz, do, dstate = eq.recurrence_backward(i["dy"], i["x"], i["forget"], cu, marks, gate=gate, reverse=reverse, dfinal=dfinal,
                                                longest=longest, with_state=True, **parts)
    torch.cuda.synchronize()
    inside = np.zeros(y.shape[0], bool)
    inside[edges[0]:edges[-1]] = True
    assert none is None and torch.equal(final, final2) and torch.equal(y[inside], y2[inside])
    for t in (y, dx, dz) + (() if gate is None else (do,)):  # rows of no sequence are left alone
        assert bool((t[~torch.from_numpy(inside).to(t.device)] == 7).all()), label
    n = lambda t: None if t is None else _np(t)  # noqa: E731
    wy, wfinal, h = stage.recurrence(n(i["x"]), n(i["forget"]), edges, n(gate), n(state), reverse)
    wdx, wdz, wdo, wds = stage.recurrence_backward(n(i["dy"]), n(i["x"]), n(i["forget"]), edges, n(gate), n(state), reverse, n(dfinal))
    M, last, before, D, Ds = _magnitudes(i, reverse, with_state, with_dfinal, h, wdx)
    eps, rel = (1e-6, 2e-6) if dtype == "f32" else (3e-6, 4e-6)
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-37
    s = inside
    z, x, dy = n(i["forget"])[s], np.abs(n(i["x"])[s]), np.abs(n(i["dy"])[s])
    f, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    bar = lambda want, work: 1.01 * (U[dtype] * np.abs(want) + work) + tiny  # noqa: E731
    factor = 1.0
    if gate is not None:
        o = n(gate)[s]
        sig = 1 / (1 + np.exp(-o))
        factor = np.abs(o) * sig
    _near(y[s], wy[s], bar(wy[s], factor * eps * M[s] + rel * np.abs(wy[s])), label + " y")
    _near(final, wfinal, eps * last + 1e-30, label + " final")
    dh = np.abs(wdx[s]) / rest
    _near(dx[s], wdx[s], bar(wdx[s], rest * eps * D[s] + rel * np.abs(wdx[s])), label + " dx")
    hx = np.abs(h[s]) + x + before[s]
    work = dh * f * rest * eps * (before[s] + hx) + f * rest * hx * eps * D[s] + rel * np.abs(wdz[s])
    _near(dz[s], wdz[s], bar(wdz[s], work), label + " dforget")
    if gate is not None:
        work = dy * sig * (1 + np.abs(o)) * (eps * M[s] + rel * np.abs(h[s]))
        _near(do[s], wdo[s], bar(wdo[s], work), label + " dgate")
    _near(dstate, wds, eps * Ds + 1e-30, label + " dstate")
    return y, final


# longest: a hint (None: unknown), which picks the form of the launch: 1 and 8 a wave a sequence, 17, 128 and 256 a workgroup with 1, 2 and 4
# groups of lanes a wave, 1000 and None of many tokens the chunks side by side, without and with a launch for the states in front of
# them. The results have to be right for each, whatever the lengths are.
@pytest.mark.parametrize("longest", [None, 1, 8, 17, 128, 256, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", list(LENS))
def test_recurrence(name, dtype, longest, cuda_device):
    lens = LENS[name]
    shift = 0 if longest is None else longest % 5  # other widths and options for each hint
    for k in range(3):
        (C, G), reverse = WIDTHS[(k + shift) % len(WIDTHS)], bool((k + shift) % 2)
        gated = bool((k + shift // 2) % 3)
        label = f"recurrence {name} C={C} G={G} {dtype} longest={longest} reverse={reverse} gated={gated}"
        print(f"[case] {label}", flush=True)
        i = _inputs(lens, C, G, dtype, cuda_device, 100 * k + len(lens), lead=3 * (k % 3), tail=5 * (k % 2), gated=gated)
        _check(i, dtype, reverse, longest, label, with_state=k % 4 != 1, with_dfinal=k % 4 != 2)


def test_chunks_beyond_the_first_rows(cuda_device):
    """A first sequence that begins thousands of rows into the tensor: chunk slots in front of it belong to none."""
    i = _inputs([900, 400], 8, 4, "bf16", cuda_device, 1, lead=3000, tail=700)
    for longest in (None, 17, 128, 256):
        _check(i, "bf16", False, longest, f"lead 3000 longest={longest}")
        _check(i, "bf16", True, longest, f"lead 3000 reverse longest={longest}")


def test_many_sequences(cuda_device):
    """More sequences than a wave's search takes in one step (64), and in two (4096), in the chunks' form too."""
    lens = [1, 0, 2, 5] * 1100
    i = _inputs(lens, 2, 1, "f32", cuda_device, 2, lead=1)
    for longest in (None, 5, 256):
        _check(i, "f32", False, longest, f"4400 sequences longest={longest}")


def test_a_sequence_of_more_chunks_than_a_join_takes_at_once(cuda_device):
    """66000 tokens (1032 chunks) beside short ones; the states are carried over the join's stages, both ways."""
    i = _inputs([3, 66000, 0, 70], 1, 2, "f32", cuda_device, 12)
    _check(i, "f32", False, None, "66000 tokens")
    _check(i, "f32", True, 20000, "66000 tokens, reverse, said to be 20000")
    _check(i, "f32", False, 2000, "66000 tokens, said to be 2000")


def test_state_in_place_and_in_pieces(cuda_device):
    """A step that updates its states in place, token by token and piece by piece, in every form of the launch; and the same bits
    every time."""
    dev = cuda_device
    for lens, C, G, longest in [([1] * 300, 24, 4, 1), ([1] * 300, 24, 4, None), ([40, 0, 3, 200], 8, 2, 17), ([700, 0, 900, 5], 33, 1, None),
                                ([700, 0, 300, 5], 32, 1, 128), ([700, 0, 300, 5], 32, 1, 256), ([700, 0, 300, 5], 32, 1, 1000), ([1, 8, 3], 6, 8, 8)]:
        i = _inputs(lens, C, G, "bf16", dev, 5)
        kw = dict(gate=i["gate"], longest=longest)
        y, final, _ = eq.recurrence(i["x"], i["forget"], i["cu"], state=i["state"], **kw)
        state = i["state"].clone()
        y2, same, _ = eq.recurrence(i["x"], i["forget"], i["cu"], state=state, final=state, **kw)
        torch.cuda.synchronize()
        assert same is state and torch.equal(y, y2) and torch.equal(final, state)
        for _ in range(3):
            y3, final3, _ = eq.recurrence(i["x"], i["forget"], i["cu"], state=i["state"], **kw)
            torch.cuda.synchronize()
            assert torch.equal(y, y3) and torch.equal(final, final3)
    # one sequence in three calls = one call
    i = _inputs([333], 16, 4, "f32", dev, 6)
    whole, final, _ = eq.recurrence(i["x"], i["forget"], i["cu"], state=i["state"], longest=333)
    state, at = i["state"].clone(), 0
    for n in (1, 131, 201):
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        y, _, _ = eq.recurrence(i["x"][at:at + n], i["forget"][at:at + n], cu, state=state, final=state, longest=n)
        torch.cuda.synchronize()
        assert float((y - whole[at:at + n]).abs().max()) <= 1e-4
        at += n
    assert float((state - final).abs().max()) <= 1e-4


def test_what_is_not_finite_stays_in_its_sequence_and_column(cuda_device):
    dev = cuda_device
    for longest in (None, 17, 256, 1000):
        i = _inputs([300, 200, 650], 8, 2, "bf16", dev, 7)
        args = dict(gate=i["gate"], longest=longest)
        run = lambda st: (*eq.recurrence(i["x"], i["forget"], i["cu"], state=st["state"], with_marks=True, **args),)  # noqa: E731
        y, final, marks = run(i)
        back = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], marks, dfinal=i["dfinal"], with_state=True, **args)
        keep = [t.clone() for t in (y, final, *back)]
        i["x"][350, 3, 1] = float("nan")
        i["x"][310, 5, 0] = float("inf")
        i["forget"][420, 1, 0] = float("nan")
        i["dy"][400, 6, 1] = float("nan")
        i["state"][1, 7, 0] = float("inf")
        i["dfinal"][1, 0, 1] = float("nan")
        y, final, marks = run(i)
        back = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], marks, dfinal=i["dfinal"], with_state=True, **args)
        torch.cuda.synchronize()
        bad = torch.zeros((8, 2), dtype=torch.bool, device=dev)
        for c, g in ((3, 1), (5, 0), (1, 0), (6, 1), (7, 0), (0, 1)):
            bad[c, g] = True
        for a, b in zip((y, final, *back), keep):
            a, b = a.clone(), b.clone()
            hit = slice(300, 500) if a.shape[0] == 1150 else slice(1, 2)
            a[hit, bad], b[hit, bad] = 0, 0
            assert torch.equal(a, b)
        assert bool(y[350:500, 3, 1].isnan().all()) and bool(y[300:350, 3, 1].isfinite().all()) and not bool(final[1, 7, 0].isfinite())


def test_extreme_gates(cuda_device):
    """Forget gates of +-infinity and of the type's largest values: all is kept, or all forgotten."""
    dev = cuda_device
    x = torch.tensor([1.0, 2.0, 3.0, 4.0], device=dev).view(4, 1, 1).repeat(1, 4, 1).to(torch.float16)
    z = torch.tensor([float("inf"), -float("inf"), 65504.0, -65504.0], device=dev).view(1, 4, 1).repeat(4, 1, 1).to(torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    h0 = torch.full((1, 4, 1), 9.0, device=dev)
    y, final, marks = eq.recurrence(x, z, cu, state=h0, with_marks=True)
    dy = torch.ones_like(x)
    dx, dz, _, dh = eq.recurrence_backward(dy, x, z, cu, marks, with_state=True)
    torch.cuda.synchronize()
    assert y[:, 0].flatten().tolist() == [9] * 4 and y[:, 2].flatten().tolist() == [9] * 4
    assert y[:, 1].flatten().tolist() == [1, 2, 3, 4] and y[:, 3].flatten().tolist() == [1, 2, 3, 4]
    assert dx[:, 0].flatten().tolist() == [0] * 4 and dx[:, 1].flatten().tolist() == [1] * 4 and not dz.any()
    dh = dh.flatten().tolist()
    assert dh[0] == 4 and dh[2] == 4 and max(abs(dh[1]), abs(dh[3])) <= 4 * 2.0 ** -126  # (half types: f is at least 2^-126)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_output_gates_of_the_lowest_and_highest_value(dtype, cuda_device):
    """silu of the type's lowest value is 0 (whatever the state), of its largest the value itself, of 0 and of large negative ones
    next to nothing; the gradients follow."""
    dev, dt = cuda_device, DT[dtype]
    top = torch.finfo(dt).max
    o = torch.tensor([-top, -top / 2, -200.0, -88.0, 0.0, 30.0], dtype=dt, device=dev).view(1, 6, 1).repeat(3, 1, 1)
    x = torch.tensor([100.0, -3.0, 0.25], device=dev).view(3, 1, 1).repeat(1, 6, 1).to(dt)
    z = torch.zeros_like(x)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=dev)
    y, _, marks = eq.recurrence(x, z, cu, gate=o, with_marks=True)
    dy = torch.ones_like(x)
    dx, dz, do, _ = eq.recurrence_backward(dy, x, z, cu, marks, gate=o)
    torch.cuda.synchronize()
    for t in (y, dx, dz, do):
        assert bool(t.isfinite().all()) and float(t[:, :4].abs().max()) <= 1e-30
    h = stage.recurrence(_np(x), _np(z), [0, 3])[0]
    assert not y[:, 4].any() and np.allclose(_np(do[:, 4]), h[:, 4] / 2, rtol=2 * U[dtype])
    assert np.allclose(_np(y[:, 5]), 30 * h[:, 5], rtol=2 * U[dtype]) and np.allclose(_np(do[:, 5]), h[:, 5], rtol=2 * U[dtype])


def test_gradients_by_differences(cuda_device):
    """Against central differences of the kernel's own forward (fp32, h = 2^-6: third-order terms of size h^2 and rounding of
    2^-24 |sum| / h, both under 1e-3 here)."""
    i = _inputs([5, 0, 9], 2, 2, "f32", cuda_device, 8)
    i["forget"] = i["forget"] * 0.3
    leaves = [i["x"].contiguous(), i["forget"].contiguous(), i["gate"].contiguous(), i["state"]]

    def loss(a, z, o, h):
        y, final, _ = eq.recurrence(a, z, i["cu"], gate=o, state=h)
        return float((y.double() * i["dy"].double()).sum() + (final.double() * i["dfinal"].double()).sum())

    _, _, marks = eq.recurrence(*leaves[:2], i["cu"], gate=leaves[2], state=leaves[3], with_marks=True)
    grads = eq.recurrence_backward(i["dy"], *leaves[:2], i["cu"], marks, gate=leaves[2], dfinal=i["dfinal"], with_state=True)
    h = 2.0 ** -6
    for k, t in enumerate(leaves):
        for e in range(0, t.numel(), 3):
            step = torch.zeros(t.numel(), device=t.device)
            step[e] = h
            up, down = (loss(*[a if j != k else t + sign * step.view(t.shape) for j, a in enumerate(leaves)]) for sign in (1, -1))
            assert abs(float(grads[k].reshape(-1)[e]) - (up - down) / (2 * h)) <= 2e-3, (k, e)


def test_offsets_past_32_bits(cuda_device):
    """Token strides that put the last rows more than 2^31 elements behind the first."""
    dev, stride, T, C = cuda_device, 1 << 22, 600, 16
    wide, outs = (torch.empty((T, stride), dtype=torch.bfloat16, device=dev) for _ in range(2))
    i = _inputs([257, T - 257], C, 1, "bf16", dev, 9)
    i["parts"] = i["parts"].contiguous()
    far = {}
    for k, name in enumerate(("x", "forget", "gate")):
        far[name] = wide[:, (k + 1) * 64:(k + 1) * 64 + C, None]
        far[name].copy_(i[name])
    for longest in (None, 17, 128, 256):
        a = eq.recurrence(i["x"], i["forget"], i["cu"], gate=i["gate"], longest=longest, with_marks=True)
        b = eq.recurrence(far["x"], far["forget"], i["cu"], gate=far["gate"], longest=longest, with_marks=True, out=outs[:, :C, None])
        da = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], a[2], gate=i["gate"], longest=longest)
        db = eq.recurrence_backward(i["dy"], far["x"], far["forget"], i["cu"], b[2], gate=far["gate"], longest=longest,
                                    dx=outs[:, 1024:1024 + C, None], dforget=outs[:, 2048:2048 + C, None])
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(p, q) for p, q in zip(da[:3], db[:3]))


def test_group_shift_streams_and_graphs(cuda_device):
    dev = cuda_device
    i = _inputs([130, 1, 40], 6, 8, "f32", dev, 10)
    roll = lambda t: t.roll(3, 2).contiguous()  # noqa: E731
    y, final, marks = eq.recurrence(i["x"], i["forget"], i["cu"], gate=i["gate"], state=i["state"], with_marks=True)
    y2, final2, _ = eq.recurrence(roll(i["x"]), roll(i["forget"]), i["cu"], gate=roll(i["gate"]), state=roll(i["state"]))
    torch.cuda.synchronize()
    assert torch.equal(y2, roll(y)) and torch.equal(final2, roll(final))
    back = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], marks, gate=i["gate"], with_state=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for longest in (None, 17, 130, 2000):
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                gy, gf, gm = eq.recurrence(i["x"], i["forget"], i["cu"], gate=i["gate"], state=i["state"], with_marks=True, longest=longest)
                gb = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], gm, gate=i["gate"], with_state=True, longest=longest)
        side.synchronize()
        for k in range(4):  # each replay against the eager result for the inputs of that time
            i["parts"].copy_(torch.randn(i["parts"].shape, generator=torch.Generator().manual_seed(k)))
            y, final, marks = eq.recurrence(i["x"], i["forget"], i["cu"], gate=i["gate"], state=i["state"], with_marks=True, longest=longest)
            back = eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], marks, gate=i["gate"], with_state=True, longest=longest)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((gy, gf, *gb), (y, final, *back)):
                assert torch.equal(a, b), (longest, k)


def test_nothing_and_refusals(cuda_device):
    dev = cuda_device
    i = _inputs([5, 3], 4, 2, "bf16", dev, 11)
    x, z, o, cu, h0 = i["x"], i["forget"], i["gate"], i["cu"], i["state"]
    none = torch.zeros((3,), dtype=torch.int32, device=dev)
    y, final, marks = eq.recurrence(x[:0], z[:0], none, state=h0, with_marks=True)
    dx, dz, _, ds = eq.recurrence_backward(y, x[:0], z[:0], none, marks, dfinal=h0, with_state=True)
    torch.cuda.synchronize()
    assert y.shape == (0, 4, 2) and torch.equal(final, h0) and torch.equal(ds, h0) and dx.shape == (0, 4, 2)
    y, final, _ = eq.recurrence(x, z, none[:1])
    assert final.shape == (0, 4, 2)
    _, _, marks = eq.recurrence(x, z, cu, gate=o, with_marks=True)
    dy = i["dy"]
    for kind, call in [
        (ValueError, lambda: eq.recurrence(x[0], z[0], cu)), (ValueError, lambda: eq.recurrence(x, z[:3], cu)),
        (ValueError, lambda: eq.recurrence(x, z.half(), cu)), (TypeError, lambda: eq.recurrence(x.double(), z.double(), cu)),
        (TypeError, lambda: eq.recurrence(x.cpu(), z, cu)), (ValueError, lambda: eq.recurrence(x, z, cu.long())),
        (ValueError, lambda: eq.recurrence(x.transpose(1, 2), z.transpose(1, 2), cu)), (ValueError, lambda: eq.recurrence(x, z, cu, state=h0[:1])),
        (ValueError, lambda: eq.recurrence(x, z, cu, state=h0.half())), (ValueError, lambda: eq.recurrence(x, z, cu, longest=-1)),
        (ValueError, lambda: eq.recurrence(x, z, cu, gate=o[:3])), (ValueError, lambda: eq.recurrence(x, z, cu[:0])),
        (eq.EqlinError, lambda: eq.recurrence(x, z, cu, out=x)), (eq.EqlinError, lambda: eq.recurrence(x, z, cu, out=x[:1].expand(8, 4, 2))),
        (ValueError, lambda: eq.recurrence_backward(dy, x, z, cu, marks[:1], gate=o)), (ValueError, lambda: eq.recurrence_backward(dy[:2], x, z, cu, marks)),
        (eq.EqlinError, lambda: eq.recurrence_backward(dy, x, z, cu, None)), (ValueError, lambda: eq.recurrence_backward(dy, x, z, cu, marks, dgate=dy)),
        (eq.EqlinError, lambda: eq.recurrence_backward(dy, x, z, cu, marks, dx=dy.clone(), dforget=x)),
    ]:
        with pytest.raises(kind):
            call()
    same = torch.empty_like(dy)
    with pytest.raises(eq.EqlinError):
        eq.recurrence_backward(dy, x, z, cu, marks, dx=same, dforget=same)
