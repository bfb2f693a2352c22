"""A forget gate of minus infinity or of the type's lowest value starts a sequence anew: f is exactly 0, so no state in front of it,
however large, has a part in what comes after, and no gradient behind it in what comes before (tolerances: none, the same bits);
its own gradient is 0."""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage as ref
from test_norm_rotary_gpu import DT, U, _np
from test_recurrence_gpu import _inputs

pytestmark = pytest.mark.gpu

LENS = [200, 1, 70]
RESET = {0: [40, 130], 1: [0], 2: [69]}  # of each sequence, its tokens with such gates


def _case(dtype, lowest, reverse, dev):
    """Inputs whose other gates remember (f = 0.9975), and the rows of the gates in question, by sequence, in the recurrence's order."""
    i = _inputs(LENS, 6, 4, dtype, dev, 3)
    i["forget"][:] = 6.0
    rows = {k: [i["edges"][k + 1] - 1 - t if reverse else i["edges"][k] + t for t in at] for k, at in RESET.items()}
    for at in rows.values():
        i["forget"][at] = lowest
    return i, rows


# the launch's forms, by the hint that picks them (test_recurrence_gpu.py)
@pytest.mark.parametrize("longest", [None, 1, 8, 17, 128, 256, 1000])
@pytest.mark.parametrize("lowest", ["lowest", "-inf"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_nothing_passes_a_gate_of_the_lowest_value(dtype, lowest, longest, cuda_device):
    low = -float("inf") if lowest == "-inf" else torch.finfo(DT[dtype]).min
    for reverse in (False, True):
        i, rows = _case(dtype, low, reverse, cuda_device)
        kw = dict(gate=i["gate"], reverse=reverse, longest=longest)
        # states of 3e38 (times 2^-126 still 3.5) in front, and none
        far, none = (eq.recurrence(i["x"], i["forget"], i["cu"], state=torch.full_like(i["state"], s), with_marks=True, **kw) for s in (3e38, 0.0))
        # the gradients of final, likewise (1e37 times 2^-126: 0.12)
        _, _, marks = eq.recurrence(i["x"], i["forget"], i["cu"], state=i["state"], with_marks=True, **kw)
        back = [eq.recurrence_backward(i["dy"], i["x"], i["forget"], i["cu"], marks, dfinal=torch.full_like(i["dfinal"], s), with_state=True, **kw)
                for s in (1e37, 0.0)]
        torch.cuda.synchronize()
        assert torch.equal(far[1], none[1]), reverse  # final
        assert torch.equal(back[0][3], back[1][3]) and not back[0][3][1].any(), reverse  # dstate
        for k, at in rows.items():
            first, last = i["edges"][k], i["edges"][k + 1]
            after = slice(first, at[0] + 1) if reverse else slice(at[0], last)
            before = slice(at[-1] + 1, last) if reverse else slice(first, at[-1])
            assert bool(none[0][after].isfinite().all()) and torch.equal(far[0][after], none[0][after]), (reverse, k)
            for a, b in zip(back[0][:3], back[1][:3]):
                assert bool(b[before].isfinite().all()) and torch.equal(a[before], b[before]), (reverse, k)


@pytest.mark.parametrize("longest", [None, 1, 17, 128, 256, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_the_gradient_of_a_gate_behind_masked_values(dtype, longest, cuda_device):
    """Tokens whose values are masked by the type's lowest value, a gate that forgets them, gradients of some hundreds behind it:
    dforget = dh (h - x) f (1 - f) is 0 there, though dh (h - x) is beyond fp32, and what it says at the masked token. Bar there: one
    rounding of the result (u), and 1e-5 for the factors (each within a few units of fp32, sums of two terms of one sign or far apart)."""
    dev, dt, low = cuda_device, DT[dtype], torch.finfo(DT[dtype]).min
    for reverse in (False, True):
        i, rows = _case(dtype, low, reverse, dev)
        gates = [r for k in (0, 2) for r in rows[k]]
        masked = [r + 1 if reverse else r - 1 for r in gates]
        i["x"][masked], i["forget"][masked] = low, 0.0
        dy = torch.full_like(i["dy"], 8.0)
        dy[masked] = 0.5
        kw = dict(reverse=reverse, longest=longest)
        _, _, marks = eq.recurrence(i["x"], i["forget"], i["cu"], state=i["state"], with_marks=True, **kw)
        dx, dz, _, dstate = eq.recurrence_backward(dy, i["x"], i["forget"], i["cu"], marks, dfinal=i["dfinal"], with_state=True, **kw)
        torch.cuda.synchronize()
        for t in (dx, dz, dstate):
            assert bool(t.isfinite().all()), reverse
        assert not dz[gates].any(), reverse
        with np.errstate(over="ignore"):  # (exp of the lowest gates' size, under a 1 /)
            want = ref.recurrence_backward(_np(dy), _np(i["x"]), _np(i["forget"]), i["edges"], None, _np(i["state"]), reverse, _np(i["dfinal"]))[1]
        want = want[masked]
        assert bool((abs(_np(dz[masked]) - want) <= (U[dtype] + 1e-5) * abs(want)).all()), reverse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_values_under_a_state_of_the_other_sign(dtype, cuda_device):
    """h - x beyond fp32 (a state of 3e37, a value of the type's lowest), dh (h - x) f (1 - f) not: the bar of the masked tokens above."""
    dev, dt = cuda_device, DT[dtype]
    x = torch.zeros((3, 6, 4), dtype=dt, device=dev)
    x[0] = torch.finfo(dt).min
    z, dy = torch.full_like(x, 2.0), torch.full_like(x, 0.25)
    cu, state = torch.tensor([0, 3], dtype=torch.int32, device=dev), torch.full((1, 6, 4), 3e37, device=dev)
    _, _, marks = eq.recurrence(x, z, cu, state=state, with_marks=True)
    _, dz, _, _ = eq.recurrence_backward(dy, x, z, cu, marks)
    torch.cuda.synchronize()
    want = ref.recurrence_backward(_np(dy), _np(x), _np(z), [0, 3], None, _np(state))[1][0]
    assert bool((abs(_np(dz[0]) - want) <= (U[dtype] + 1e-5) * abs(want)).all())
