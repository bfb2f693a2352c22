"""GPU tests of the fp16 attention gradients at both ends of the type's range. Probabilities and score gradients are operands of
products in fp16 (normal from 2^-14 to 65504); they keep the type's 11 bits whatever the size of d_o, the number of keys and
the score gradients themselves, so the bars are those of test_attention_gpu.py with the results' own subnormal rounding
(half a step, 2^-25 an element) added."""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage
from test_attention_gpu import U, _inputs, _np, _terms

pytestmark = pytest.mark.gpu


def _check(grads, do, q, k, v, cu_q, cu_k, label, **kw):
    args = [_np(t) for t in (do, q, k, v)] + [cu_q.tolist(), cu_k.tolist()]
    u, tiny = U["f16"], 2.0 ** -25
    for name, g, w, t in zip(("dq", "dk", "dv"), grads, stage.attention_backward(*args, **kw), _terms(*args, **kw)):
        assert np.abs(w).max() < 65504, "the exact gradient has to be in range"
        g = _np(g)
        d, bar = np.linalg.norm(g - w), 3 * u * np.linalg.norm(w) + 1e-5 * np.linalg.norm(t) + tiny * np.sqrt(w.size)
        dm, bm = np.abs(g - w).max(), 8 * u * np.abs(w).max() + 2e-5 * np.abs(t).max() + tiny
        print(f"[parity] {label} {name}: norm {d:.2e} of {bar:.2e}, max {dm:.2e} of {bm:.2e} (largest {np.abs(w).max():.2e})", flush=True)
        assert np.isfinite(g).all() and d <= bar and dm <= bm, (label, name)


def _run(q, k, v, do, cu_q, cu_k, label, **kw):
    print(f"[case] {label}", flush=True)
    o, lse = eq.attention(q, k, v, cu_q, cu_k, **kw)
    grads = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, **kw)
    torch.cuda.synchronize()
    _check(grads, do, q, k, v, cu_q, cu_k, label, **kw)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("size", [1e-2, 1e-4, 1e-5])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_small_gradients_over_many_keys(D, size, causal, cuda_device):
    """Score gradients of about size sqrt(D) / 3000: below fp16's subnormal step for the smallest."""
    lens = [3000, 40]
    q, k, v, do, cu, _ = _inputs(lens, lens, 4, 1, D, "f32", cuda_device, seed=31)
    q, k, v, do = q.half(), k.half(), v.half(), (do * size).half()
    _run(q, k, v, do, cu, cu, f"small D={D} {size} causal={causal}", causal=causal)


@pytest.mark.parametrize("D", [32, 64, 128])
def test_large_gradients(D, cuda_device):
    """d_o of about 10^4 (a large loss scale): dP - delta exceeds 65504 while every gradient is in range."""
    lens = [16, 9, 100, 2]
    q, k, v, do, cu, _ = _inputs(lens, lens, 2, 2, D, "f32", cuda_device, seed=32)
    q, k, v, do = (3 * q).half(), (3 * k).half(), (4 * v).half(), (1e4 * do).clamp(-6e4, 6e4).half()
    for causal in (False, True):
        _run(q, k, v, do, cu, cu, f"large D={D} causal={causal}", scale=0.01, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
def test_sizes_that_grow_and_shrink_from_tile_to_tile(D, cuda_device):
    """Rows whose d_o, and keys whose values, run from 2^-12 to 2^8 and back from one tile of 32 to the next, smallest first and
    largest first: each row's and each key's sums are carried by the largest."""
    n = 700
    q, k, v, do, cu, _ = _inputs([n], [n], 2, 1, D, "f32", cuda_device, seed=33)
    for turn in (1, -1):
        ramp = 2.0 ** (turn * (10 * torch.sin(torch.arange(n, device=cuda_device) // 32 * 0.7)) - 2)
        a, b = (v * ramp[:, None, None]).half(), (do * ramp.flip(0)[:, None, None]).half()
        _run(q.half(), k.half(), a, b, cu, cu, f"ramp D={D} {turn}", scale=0.03)


def test_probabilities_of_many_keys(cuda_device):
    """128 rows over 100000 keys: probabilities of about 10^-5, below fp16's normal range, as operands of dv."""
    q, k, v, do, cu_q, cu_k = _inputs([128], [100000], 1, 1, 64, "f16", cuda_device, seed=34)
    _run(q, k, v, do, cu_q, cu_k, "many keys")


def test_infinite_and_nan_rows_stay_where_they_are(cuda_device):
    """A row of infinities in d_o makes its own gradients and those of the keys that it sees infinite or NaN, nothing else."""
    lens = [150, 90]
    q, k, v, do, cu, _ = _inputs(lens, lens, 2, 1, 64, "f16", cuda_device, seed=35)
    o, lse = eq.attention(q, k, v, cu, cu, causal=True)
    clean = eq.attention_backward(do, q, k, v, o, lse, cu, cu, causal=True)
    for bad in (float("inf"), float("nan")):
        do2 = do.clone()
        do2[100] = bad
        dq, dk, dv = eq.attention_backward(do2, q, k, v, o, lse, cu, cu, causal=True)
        torch.cuda.synchronize()
        keep = torch.ones(240, dtype=torch.bool)
        keep[100] = False
        assert torch.equal(dq[keep], clean[0][keep]) and not bool(dq[100].isfinite().any())
        for a, b in ((dk, clean[1]), (dv, clean[2])):
            assert torch.equal(a[101:], b[101:]) and not bool(a[:101].isfinite().any())


@pytest.mark.parametrize("D", [32, 64, 128])
def test_scores_in_the_millions(D, cuda_device):
    """Scores up to 2^25 in log2 units, where fp32's step is 2: half a step in the score, in the maximum, in lse and in its way
    back, and the constants' own roundings, leave exp(score - lse) of the one key that matters anywhere up to 2^5, above 1
    and still far inside the type's range. Bar: every gradient is finite, and dv within that factor of the sum of |d_o|."""
    q, k, v, do, cu, _ = _inputs([70], [70], 2, 1, D, "f32", cuda_device, seed=36)
    q, k, v, do = (100 * q).half(), (100 * k).half(), v.half(), do.half()
    scale = 600 * D ** -0.5
    o, lse = eq.attention(q, k, v, cu, cu, scale=scale)
    assert 1e7 < float(lse.abs().max()) < 2.3e7
    dq, dk, dv = eq.attention_backward(do, q, k, v, o, lse, cu, cu, scale=scale)
    torch.cuda.synchronize()
    assert all(bool(t.isfinite().all()) for t in (o, lse, dv))
    assert float(dv.float().abs().max()) <= 32 * float(do.float().abs().sum(dim=(0, 1)).max())
