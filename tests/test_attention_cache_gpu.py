"""GPU parity of eqlin_attention where single tokens, short runs of tokens and whole prompts are in one call over
caches of every length, and where a tensor is longer than 32 bits of offset. Bars as in test_attention_gpu.py."""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage
from test_attention_gpu import DT, _check_forward, _check_grads, _inputs, _np

pytestmark = pytest.mark.gpu

# (query lengths, key lengths, Hq, Hkv, D)
MIXED = {
    # tokens over caches next to prompts, shorter and longer than a chunk's room of 32 rows, and nothing at all
    "steps_and_prompt": ([1] * 12 + [130, 0, 1], [900] * 6 + [1, 2, 31, 33, 0, 2000] + [130, 70, 600], 4, 1, 128),
    "room_ends": ([7, 8, 9, 1, 1], [700, 700, 700, 40, 1300], 4, 1, 64),
    "odd_group": ([4, 7, 1, 40], [513, 800, 1025, 640], 15, 3, 40),
    # no more tokens than sequences, but several of them in one
    "empty_but_one": ([0, 0, 0, 0, 5, 0], [500, 0, 300, 700, 900, 64], 8, 2, 64),
    "many_rows_in_one": ([0] * 39 + [40], [300] * 39 + [520], 2, 1, 32),
    # the prompt itself over a long cache: its keys split as well, rows that see nothing among them
    "piece_of_a_prompt": ([1, 1, 70, 1], [2000, 1500, 2500, 10], 2, 2, 128),
    "more_queries_than_keys": ([50, 1, 2], [20, 3000, 1], 2, 2, 64),
    # more heads than a product has columns
    "group_of_40": ([1, 2], [700, 300], 40, 1, 64),
    "group_of_32": ([1, 1, 3], [700, 300, 2000], 32, 1, 64),
    # enough sequences and heads for a workgroup each
    "many_steps": ([1] * 63 + [2], [240 + i for i in range(64)], 16, 8, 32),
    "two_levels_of_search": ([1] * 150, [3 + 5 * (i % 7) for i in range(149)] + [60000], 2, 1, 64),
}


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", MIXED)
def test_attention_steps_and_prompts(name, dtype, causal, cuda_device):
    lq, lk, Hq, Hkv, D = MIXED[name]
    label = f"{name} {dtype} causal={causal}"
    print(f"[case] {label}", flush=True)
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, Hq, Hkv, D, dtype, cuda_device, seed=11)
    o = torch.full_like(q, float("nan"))
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=causal, out=o)
    torch.cuda.synchronize()
    _check_forward(o, lse, q, k, v, cu_q, cu_k, dtype, label, causal=causal)


@pytest.mark.parametrize("name", ["steps_and_prompt", "piece_of_a_prompt", "empty_but_one"])
def test_attention_steps_and_prompts_repeat(name, cuda_device):
    """The same bits every time, whatever the workspace holds."""
    lq, lk, Hq, Hkv, D = MIXED[name]
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, Hq, Hkv, D, "bf16", cuda_device, seed=12)
    ws = torch.full((1 << 26,), 0xff, dtype=torch.uint8, device=cuda_device)
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
    for fill in (0xff, 0, 0x7f):
        ws.fill_(fill)
        o2, lse2 = eq.attention(q, k, v, cu_q, cu_k, causal=True, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_values_of_later_tokens_in_a_step(dtype, cuda_device):
    """Infinities and NaN in keys that a causal row of a short run does not see stay out of its result."""
    dev, lq, lk = cuda_device, [3, 1, 60, 1], [900, 700, 800, 40]
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, 4, 2, 64, dtype, dev, seed=13)
    clean, _ = eq.attention(q, k, v, cu_q, cu_k, causal=True)
    at = 899  # seen by the first sequence's last token alone
    v[at] = float("inf")
    k[at] = float("nan")
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
    torch.cuda.synchronize()
    assert torch.equal(o[:2], clean[:2]) and torch.equal(o[3:], clean[3:])
    assert bool(o[2].isnan().all())


@pytest.mark.parametrize("lens", [([1, 2], [2600, 1600]), ([70, 9], [2600, 1600])], ids=["step", "prompt"])
def test_attention_offsets_beyond_32_bits(lens, cuda_device):
    """Tokens 2^20 elements apart: the last ones' offsets need 33 bits (two buffers of 9 GB, of which only the heads are touched)."""
    dev, (lq, lk) = cuda_device, lens
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, 4, 2, 64, "bf16", dev, seed=14)
    stride, n = 1 << 20, sum(lk)
    kv, grad = (torch.empty((n * stride,), dtype=DT["bf16"], device=dev) for _ in range(2))
    kb, vb, dkb, dvb = (t.as_strided((n, 2, 64), (stride, 64, 1), at) for t in (kv, grad) for at in (0, 1024))
    kb.copy_(k)
    vb.copy_(v)
    o, lse = eq.attention(q, kb, vb, cu_q, cu_k, causal=True)
    grads = eq.attention_backward(do, q, kb, vb, o, lse, cu_q, cu_k, causal=True, dk=dkb, dv=dvb)
    torch.cuda.synchronize()
    _check_forward(o, lse, q, k, v, cu_q, cu_k, "bf16", f"far {lq}", causal=True)
    _check_grads([g.contiguous() for g in grads], do, q, k, v, cu_q, cu_k, "bf16", f"far {lq}", causal=True)


def test_attention_outputs_that_fold(cuda_device):
    dev = cuda_device
    q, k, v, do, cu_q, cu_k = _inputs([10], [12], 4, 4, 32, "bf16", dev)
    o, lse = eq.attention(q, k, v, cu_q, cu_k)
    flat = torch.zeros((4096,), dtype=torch.bfloat16, device=dev)
    for strides in ((128, 16, 1), (16, 32, 1), (0, 32, 1), (128, 0, 1)):
        with pytest.raises(eq.EqlinError):
            eq.attention(q, k, v, cu_q, cu_k, out=flat.as_strided((10, 4, 32), strides))
        with pytest.raises(eq.EqlinError):
            eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, dk=flat.as_strided((12, 4, 32), strides))
    same = torch.empty_like(k)
    with pytest.raises(eq.EqlinError):
        eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, dk=same, dv=same)


def test_attention_gradients_of_a_causal_sequences_first_rows(cuda_device):
    """The first rows of a causal sequence carry much of dq's and dk's norm; their delta takes no part of o's rounding.

    Bar: a value's rounding is uniform in half a step; over a logarithmically spread significand its relative rms is
    u sqrt(E[1/m^2] / 3) = 0.425 u. dq and dk have two such, dS's and their own: 0.601 u. delta of rows past 64 keys, from
    the rounded o, adds at most (1 / sqrt(D) + 1 / sqrt(24)) of one (an even softmax of normal scores over 64 keys weighs
    like 24): sqrt(2 + 0.085) 0.425 u = 0.613 u; 0.64 u leaves room for the draw."""
    lens = [200, 150, 199, 65, 130, 180]
    q, k, v, do, cu, _ = _inputs(lens, lens, 2, 2, 128, "bf16", cuda_device, seed=15)
    o, lse = eq.attention(q, k, v, cu, cu, causal=True)
    grads = eq.attention_backward(do, q, k, v, o, lse, cu, cu, causal=True)
    torch.cuda.synchronize()
    want = stage.attention_backward(*(_np(t) for t in (do, q, k, v)), cu.tolist(), cu.tolist(), causal=True)
    for name, g, w in zip(("dq", "dk"), grads, want):
        err = np.linalg.norm(_np(g) - w) / np.linalg.norm(w)
        print(f"[parity] {name}: {err / 2 ** -8:.3f} u", flush=True)
        assert err <= 0.64 * 2 ** -8, name


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_gradients_of_few_rows(dtype, cuda_device):
    """Few workgroups: dq's keys and dk's and dv's rows are split, with lengths that leave some parts empty."""
    dev = cuda_device
    for lq, lk, Hq, Hkv, D in (([40, 0, 7], [900, 30, 700], 4, 2, 64), ([300], [1100], 2, 1, 128), ([70, 500], [70, 20], 1, 1, 40)):
        label = f"few {lq} {lk} {dtype}"
        print(f"[case] {label}", flush=True)
        q, k, v, do, cu_q, cu_k = _inputs(lq, lk, Hq, Hkv, D, dtype, dev, seed=16)
        o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
        grads = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=True)
        torch.cuda.synchronize()
        _check_forward(o, lse, q, k, v, cu_q, cu_k, dtype, label, causal=True)
        _check_grads(grads, do, q, k, v, cu_q, cu_k, dtype, label, causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_gradients_of_rows_before_a_bad_key(dtype, cuda_device):
    """A causal row's dq has no part of what later keys hold, where its keys are split into ranges too."""
    q, k, v, do, cu_q, cu_k = _inputs([300], [1100], 4, 2, 64, dtype, cuda_device, seed=17)
    run = lambda: (lambda o, lse: (o, eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=True)[0]))(  # noqa: E731
        *eq.attention(q, k, v, cu_q, cu_k, causal=True))
    o, dq = run()
    k[1050] = float("nan")  # row 250 is the first to see it
    v[1050] = float("inf")
    o2, dq2 = run()
    torch.cuda.synchronize()
    assert torch.equal(o[:250], o2[:250]) and torch.equal(dq[:250], dq2[:250])
    assert bool(o2[250:].isnan().all()) and bool(dq2[250:].isnan().all())
