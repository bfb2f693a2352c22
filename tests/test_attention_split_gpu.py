"""GPU tests of the attention gradients where a launch too small to fill the card is split (dq's keys into ranges, the rows of
dk's and dv's key tiles into shares): rows that belong to no sequence, and delta of rows that see few keys. Bars as in
test_attention_gpu.py."""
import ctypes

import pytest
import torch

import fourier_domain_linear_amd as eq
from test_attention_gpu import DT, _check_grads, _cu, _inputs

pytestmark = pytest.mark.gpu


def _splits(q, k, v, o, lse, cu_q, cu_k, causal):
    """Whether the gradients of this call are split: their workspace holds more than one value a row."""
    a = eq._attention_args(q, k, v, o, lse, cu_q, cu_k, None, causal, None)[0]
    return eq.load_library().eqlin_attention_backward_workspace(ctypes.byref(a)) > 4 * (q.shape[0] * q.shape[1] + 64)


# (lengths, Hq, Hkv, D, whether the gradients are split)
OUTSIDE = {
    "one_long": ([1500], 2, 1, 64, True),
    "ragged": ([900, 0, 64, 700], 4, 4, 40, True),
    "step": ([1], 4, 2, 128, True),
    "many": ([100] * 100, 16, 8, 32, False),
}


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", OUTSIDE)
def test_rows_outside_every_sequence_are_not_written(name, dtype, causal, cuda_device):
    """Tensors of a fixed capacity: rows in front of the first sequence and behind the last keep what they hold, in o and in
    every gradient, whatever the workspace holds; the sequences' own rows are those of tensors without such rows."""
    lens, Hq, Hkv, D, split = OUTSIDE[name]
    print(f"[case] {name} {dtype} causal={causal}", flush=True)
    front, back, n = 3, 70, sum(lens)
    q, k, v, do, cu, _ = _inputs(lens, lens, Hq, Hkv, D, dtype, cuda_device, seed=21)
    room = lambda t, fill: torch.cat([torch.full_like(t[:1], fill).expand(r, -1, -1) if r else t for r in (front, 0, back)])  # noqa: E731
    q2, k2, v2, do2 = (room(t, float("nan")) for t in (q, k, v, do))
    cu2 = cu + front
    ws = torch.full((1 << 27,), 0xff, dtype=torch.uint8, device=cuda_device)
    out = torch.full_like(q2, 7.0)
    o, lse = eq.attention(q, k, v, cu, cu, causal=causal)
    o2, lse2 = eq.attention(q2, k2, v2, cu2, cu2, causal=causal, out=out, workspace=ws)
    assert _splits(q2, k2, v2, o2, lse2, cu2, cu2, causal) == split
    grads = [torch.full_like(t, 7.0) for t in (q2, k2, v2)]
    for fill in (0xff, 0x3f):
        ws.fill_(fill)
        eq.attention_backward(do2, q2, k2, v2, o2, lse2, cu2, cu2, causal=causal, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
        torch.cuda.synchronize()
        for what, t in zip(("o", "dq", "dk", "dv"), (out, *grads)):
            rows = torch.cat([t[:front], t[front + n:]])
            assert bool((rows == 7.0).all()), (what, fill)
        _check_grads([g[front:front + n] for g in grads], do, q, k, v, cu, cu, dtype, f"outside {name} {dtype}", causal=causal)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_key_has_no_score_gradient_in_a_split_launch(dtype, causal, cuda_device):
    """Softmax over one key is 1 whatever the score, so sequences of one key leave dq and dk at zero, to the bit, next to one
    that splits the launch too; so does a causal sequence whose first row alone has a gradient."""
    lens = [1, 1, 2600, 1]
    q, k, v, do, cu, _ = _inputs(lens, lens, 4, 2, 64, dtype, cuda_device, seed=22)
    o, lse = eq.attention(q, k, v, cu, cu, causal=causal)
    assert _splits(q, k, v, o, lse, cu, cu, causal)
    dq, dk, dv = eq.attention_backward(do, q, k, v, o, lse, cu, cu, causal=causal)
    torch.cuda.synchronize()
    short = [0, 1, sum(lens) - 1]
    assert not dq[short].any() and not dk[short].any() and dv[short].any()
    if causal:
        do[3:sum(lens) - 1] = 0  # (the long sequence's rows but its first)
        dq, dk, dv = eq.attention_backward(do, q, k, v, o, lse, cu, cu, causal=True)
        torch.cuda.synchronize()
        assert not dq.any() and not dk.any() and dv[2].any()


@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (8, 8)], ids=["h1", "h2on1", "h8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_delta_of_first_rows_in_a_split_launch(dtype, heads, cuda_device):
    """The first 64 rows of a causal sequence of 2048 alone have a gradient, and all values have a large common part: dP - delta
    is then small against delta, and a delta from the rounded o would be off by u |o| |dO|, many times the bars. delta of
    rows that see no key past the first tile comes from the tile's own probabilities, for dk as well as for dq."""
    n, D, (Hq, Hkv) = 2048, 128, heads
    q, k, v, do, cu, _ = _inputs([n], [n], Hq, Hkv, D, dtype, cuda_device, seed=23)
    v = (8 + v / 4).to(DT[dtype])
    do[64:] = 0
    o, lse = eq.attention(q, k, v, cu, cu, causal=True)
    assert _splits(q, k, v, o, lse, cu, cu, True)
    grads = eq.attention_backward(do, q, k, v, o, lse, cu, cu, causal=True)
    torch.cuda.synchronize()
    assert not any(bool(g[64:].any()) for g in grads)
    first = _cu([64], cuda_device)
    _check_grads([g[:64] for g in grads], do[:64], q[:64], k[:64], v[:64], first, first, dtype, f"first rows {dtype} {heads}", causal=True)
