"""eqlin_recurrence and its backward where one operand alone keeps a lane from two columns at once: an odd token stride, a first
element or a state off two elements. The width is even, so every clause of that choice is met by itself.

With strides odd everywhere the results are held against the fp64 oracle (bars: test_recurrence_gpu.py); with one operand odd the
same kernel runs, so they are the same bits; with none odd the lanes take pairs, again against the oracle."""
import ctypes

import pytest
import torch

import fourier_domain_linear_amd as eq
from test_norm_rotary_gpu import DT
from test_recurrence_gpu import _check, _inputs

pytestmark = pytest.mark.gpu

LENS, C, G = [150, 0, 1, 90], 17, 2
ROWS_IN, ROWS_OUT = ("x", "forget", "gate", "dy"), ("y", "dx", "dforget", "dgate")
STATES_IN, STATES_OUT = ("state", "dfinal"), ("final", "dstate", "marks")


def _place(t, stride, offset):
    """t's rows, `stride` elements apart, from element `offset` of a buffer on (states: stride = their own)."""
    n = t.shape[0]
    buf = torch.full((max(n, 1) * stride + offset,), 7.0, dtype=t.dtype, device=t.device)
    view = buf.as_strided(t.shape, (stride, G, 1), offset)
    view.copy_(t)
    return view


def _call(ops, cu, reverse, longest, dtype):
    """Forward and backward through the C entry points with the given tensors."""
    lib, T = eq.load_library(), ops["x"].shape[0]
    p = lambda n: ops[n].data_ptr()  # noqa: E731
    s = lambda n: ops[n].stride(0)  # noqa: E731
    a = eq.RecurrenceArgs(p("x"), p("forget"), p("gate"), p("y"), p("state"), p("final"), p("marks"), s("x"), s("forget"), s("gate"), s("y"),
                          cu.data_ptr(), T, longest or 0, len(LENS), C, G, int(reverse), eq._dtype_code(DT[dtype]))
    g = eq.RecurrenceGrads(p("dy"), p("dfinal"), p("dx"), p("dforget"), p("dgate"), p("dstate"), s("dy"), s("dx"), s("dforget"), s("dgate"))
    stream = torch.cuda.current_stream().cuda_stream
    for need, call in ((lib.eqlin_recurrence_workspace(ctypes.byref(a)), lambda w, n: lib.eqlin_recurrence(ctypes.byref(a), w, n, stream)),
                       (lib.eqlin_recurrence_backward_workspace(ctypes.byref(a)),
                        lambda w, n: lib.eqlin_recurrence_backward(ctypes.byref(a), ctypes.byref(g), w, n, stream))):
        ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=cu.device)
        assert call(ws.data_ptr(), need) == 0, lib.eqlin_last_error()
        torch.cuda.synchronize()
    return {n: ops[n].clone() for n in ROWS_OUT + ("final", "dstate")}


@pytest.mark.parametrize("longest", [None, 1, 8, 17, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_operand_off_pairs(dtype, longest, cuda_device):
    dev, L, reverse = cuda_device, C * G, longest == 17
    print(f"[case] {dtype} longest={longest}", flush=True)
    i = _inputs(LENS, C, G, dtype, dev, 21)
    _check(i, dtype, reverse, longest, f"pairs {dtype} longest={longest}")
    odd = {**i, **{n: _place(i[n], 3 * L + 1, 1) for n in ("x", "forget", "gate")}}
    _check(odd, dtype, reverse, longest, f"odd strides {dtype} longest={longest}")

    T, B = i["x"].shape[0], len(LENS)
    rows = {n: i[n].contiguous() if n in i else torch.full_like(i["dy"], 7.0) for n in ROWS_IN + ROWS_OUT}
    states = {n: i[n] if n in i else torch.full((eq.recurrence_marks(T, B) if n == "marks" else B, C, G), 7.0, device=dev) for n in STATES_IN + STATES_OUT}
    fresh = lambda: {n: t.clone() for n, t in {**rows, **states}.items()}  # noqa: E731

    def run(change):
        return _call({**fresh(), **change}, i["cu"], reverse, longest, dtype)

    want = run({n: _place(t, L + 1, 0) for n, t in rows.items()})
    single = []
    for n, t in rows.items():
        single += [(n, "stride", _place(t, L + 1, 0)), (n, "offset", _place(t, L + 2, 1))]
    single += [(n, "offset", _place(t, L, 1)) for n, t in states.items()]
    # (operands of one direction keep that one from pairs; with x, forget, gate and marks it is both)
    ways = {"y": "f", "state": "f", "final": "f", "x": "fb", "forget": "fb", "gate": "fb", "marks": "fb"}
    results = {"f": ("y", "final"), "b": ("dx", "dforget", "dgate", "dstate")}
    for n, what, t in single:
        got = run({n: t})
        for way in ways.get(n, "b"):
            for name in results[way]:
                assert torch.equal(got[name], want[name]), (n, what, name)
