"""GPU parity of eqlin_attention and its backward with the fp64 oracle (oracle/stage.py) on the same rounded
inputs, at the lengths, head layouts, strides and masks where such kernels go wrong.

Bars, from the arithmetic (u = the unit roundoff: bf16 2^-8, fp16 2^-11, fp32 2^-24):
* o, each element: one rounding of the result and one of each probability -> u |o| + u sum p |v|, plus the fp32
  part (scores, exponentials and sums over up to a few thousand terms) 2e-6 sum p |v|, plus for fp16 half a
  subnormal step a probability, 2^-25 sum |v|; all times 1.01 for the bounds' own second-order terms.
* lse: 2e-6 (1 + |lse|), fp32.
* gradients: Frobenius. Rounded probabilities or score gradients, the rounded result, and delta from the rounded
  o: three independent roundings of rms u / sqrt 3 or less, bound 3 u of the result; the largest element error is
  bounded by 8 u of the largest element. The fp32 part is relative to the terms before dP - delta cancels
  (scale sum p (|dP| + |delta|) |k| for dq, the transpose for dk, sum p |do| for dv): 1e-5 of their norm, 2e-5 of
  their largest. (A token that sees one key has exactly dq = 0, by that cancellation alone.)
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


def _cu(lens, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def _inputs(lq, lk, Hq, Hkv, D, dtype, dev, seed=0):
    gen = torch.Generator().manual_seed(seed)
    draw = lambda n, h: torch.randn((n, h, D), generator=gen).to(DT[dtype]).to(dev)  # noqa: E731
    q, k, v, do = draw(sum(lq), Hq), draw(sum(lk), Hkv), draw(sum(lk), Hkv), draw(sum(lq), Hq)
    return q, k, v, do, _cu(lq, dev), _cu(lk, dev)


def _check_forward(o, lse, q, k, v, cu_q, cu_k, dtype, label, **kw):
    args = [_np(t) for t in (q, k, v)]
    cu = [t.tolist() for t in (cu_q, cu_k)]
    kw = {n: (x.tolist() if isinstance(x, torch.Tensor) else x) for n, x in kw.items()}
    want, want_lse = stage.attention(*args, *cu, **kw)
    mag, _ = stage.attention(args[0], args[1], np.abs(args[2]), *cu, **kw)
    u = U[dtype]
    bar = 1.01 * (u * np.abs(want) + (u + 2e-6) * mag) + 1e-30
    if dtype == "f16":
        for i in range(len(cu[0]) - 1):
            grp = q.shape[1] // k.shape[1]
            total = np.abs(args[2][cu[1][i]:cu[1][i + 1]]).sum(0)
            bar[cu[0][i]:cu[0][i + 1]] += 2.0 ** -25 * np.repeat(total, grp, axis=0)[None]
    got, got_lse = _np(o), _np(lse)
    d = np.abs(got - want)
    worst = float((d / bar).max()) if d.size else 0.0
    print(f"[parity] {label}: o worst {worst:.3f} of the bar", flush=True)
    assert np.isfinite(got).all() and worst <= 1.0, label
    empty = np.isneginf(want_lse)
    assert np.array_equal(empty, np.isneginf(got_lse)), label
    dl = np.abs(got_lse[~empty] - want_lse[~empty])
    assert (dl <= 2e-6 * (1 + np.abs(want_lse[~empty]))).all(), (label, dl.max() if dl.size else 0)
    assert not got[empty].any(), label


def _terms(do, q, k, v, cu_q, cu_k, causal=False, scale=None, len_k=None):
    """What dq, dk and dv are sums of, without signs and before dP - delta cancels."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    grp = q.shape[1] // k.shape[1]
    for rq, rk, lq, lk in stage._sequences(cu_q, cu_k, len_k):
        for h in range(q.shape[1]):
            g = h // grp
            p, _ = stage._softmax(q[rq, h] @ k[rk, g].T * scale, stage._see(lq, lk, causal))
            dp = np.abs(do[rq, h]) @ np.abs(v[rk, g]).T
            ds = p * (dp + (p * dp).sum(axis=1, keepdims=True)) * scale
            dv[rk, g] += p.T @ np.abs(do[rq, h])
            dq[rq, h] = ds @ np.abs(k[rk, g])
            dk[rk, g] += ds.T @ np.abs(q[rq, h])
    return dq, dk, dv


def _check_grads(grads, do, q, k, v, cu_q, cu_k, dtype, label, **kw):
    kw = {n: (x.tolist() if isinstance(x, torch.Tensor) else x) for n, x in kw.items()}
    args = [_np(t) for t in (do, q, k, v)] + [cu_q.tolist(), cu_k.tolist()]
    u = U[dtype]
    for name, g, w, t in zip(("dq", "dk", "dv"), grads, stage.attention_backward(*args, **kw), _terms(*args, **kw)):
        g = _np(g)
        d, bar = np.linalg.norm(g - w), 3 * u * np.linalg.norm(w) + 1e-5 * np.linalg.norm(t)
        dm, bm = np.abs(g - w).max(initial=0.0), 8 * u * np.abs(w).max(initial=0.0) + 2e-5 * np.abs(t).max(initial=0.0)
        print(f"[parity] {label} {name}: norm {d:.2e} of {bar:.2e}, max {dm:.2e} of {bm:.2e}", flush=True)
        assert np.isfinite(g).all() and d <= bar and dm <= bm, (label, name, d, bar, dm, bm)


# (query lengths, key lengths, Hq, Hkv, D): lengths of zero and one, tiles cut short, several tiles, grouped
# heads with odd groups, every padding of D, more queries than keys, few rows over many keys (split over keys)
CASES = [
    ([1], [1], 1, 1, 8),
    ([64], [64], 2, 2, 32),
    ([0, 5, 0, 1], [3, 0, 0, 7], 3, 3, 40),
    ([196, 49, 1, 63], [196, 49, 1, 63], 4, 4, 128),
    ([130, 257], [130, 257], 6, 2, 64),
    ([33, 100], [300, 100], 5, 1, 96),
    ([70, 3], [20, 3], 4, 4, 64),
    ([1, 1, 1], [1000, 7, 513], 8, 1, 128),
    ([1], [5000], 4, 4, 64),
    ([4, 1], [2049, 1], 12, 3, 24),
    ([40], [3000], 7, 7, 128),
    ([17] * 70, [17] * 70, 2, 1, 16),
    ([3] * 70 + [200], [9] * 70 + [201], 2, 2, 72),
]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[f"c{i}" for i in range(len(CASES))])
def test_attention(case, dtype, causal, cuda_device):
    lq, lk, Hq, Hkv, D = case
    label = f"attention q={lq[:4]} k={lk[:4]} Hq={Hq} Hkv={Hkv} D={D} {dtype} causal={causal}"
    print(f"[case] {label}", flush=True)
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, Hq, Hkv, D, dtype, cuda_device)
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    _check_forward(o, lse, q, k, v, cu_q, cu_k, dtype, label, causal=causal)
    grads = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=causal)
    torch.cuda.synchronize()
    _check_grads(grads, do, q, k, v, cu_q, cu_k, dtype, label, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 150], ids=["step", "prompt"])
def test_attention_cache_with_room(rows, dtype, cuda_device):
    """len_k: keys past each length hold NaN and infinity and have no part; their gradients are zeros."""
    dev = cuda_device
    lq, room, used = [rows, 2, 1, 4], [700, 64, 128, 33], [651, 0, 128, 5]
    q, k, v, do, cu_q, cu_k = _inputs(lq, room, 6, 2, 64, dtype, dev, seed=1)
    len_k = torch.tensor(used, dtype=torch.int32, device=dev)
    for i, (r, n) in enumerate(zip(room, used)):
        at = sum(room[:i])
        k[at + n:at + r] = float("nan")
        v[at + n:at + r] = float("inf")
    for causal in (False, True):
        label = f"cache rows={rows} {dtype} causal={causal}"
        print(f"[case] {label}", flush=True)
        o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=causal, len_k=len_k)
        grads = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=causal, len_k=len_k)
        torch.cuda.synchronize()
        kz, vz = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
        _check_forward(o, lse, q, kz, vz, cu_q, cu_k, dtype, label, causal=causal, len_k=len_k)
        _check_grads(grads, do, q, kz, vz, cu_q, cu_k, dtype, label, causal=causal, len_k=len_k)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_of_a_qkv_layer_output(dtype, cuda_device):
    """q, k and v as strided views of one [N, C, G] tensor (heads of 8 channels x G = 8), o and the gradients
    into views too; a shift of the group axis commutes with the operator."""
    dev, lens, H, dc, G = cuda_device, [60, 131], 4, 8, 8
    gen = torch.Generator().manual_seed(5)
    y = torch.randn((sum(lens), 3 * H * dc, G), generator=gen).to(DT[dtype]).to(dev)
    do = torch.randn((sum(lens), H, dc, G), generator=gen).to(DT[dtype]).to(dev)
    cu = _cu(lens, dev)
    parts = lambda t: t.view(t.shape[0], 3 * H, dc, G).split(H, 1)  # noqa: E731
    q, k, v = parts(y)
    out = torch.full((sum(lens), 2 * H, dc, G), 7.0, dtype=DT[dtype], device=dev)
    o, lse = eq.attention(q, k, v, cu, cu, out=out[:, H:])
    grad = torch.full_like(y, float("nan"))
    dq, dk, dv = parts(grad)
    eq.attention_backward(do, q, k, v, o, lse, cu, cu, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    assert bool((out[:, :H] == 7.0).all())
    flat = [t.reshape(t.shape[0], H, dc * G) for t in (q, k, v)]
    _check_forward(o.reshape(-1, H, dc * G), lse, *flat, cu, cu, dtype, f"views {dtype}")
    _check_grads([t.reshape(-1, H, dc * G) for t in (dq, dk, dv)], do.reshape(-1, H, dc * G), *flat, cu, cu, dtype, f"views {dtype}")
    q2, k2, v2 = parts(y.roll(3, 2).contiguous())
    o2, lse2 = eq.attention(q2, k2, v2, cu, cu)
    torch.cuda.synchronize()
    # the same sums with the head's entries permuted: fp32 order and one rounding apart
    assert float((o2.double() - o.roll(3, 3).double()).norm() / o.double().norm()) <= 2 * U[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [24, 64, 128])
def test_attention_one_key_has_no_score_gradient(D, dtype, cuda_device):
    """Softmax over one key is 1 whatever the score: dq and dk are zeros, to the bit."""
    q, k, v, do, cu_q, cu_k = _inputs([1, 1, 5], [1, 1, 1], 4, 2, D, dtype, cuda_device, seed=8)
    o, lse = eq.attention(q, k, v, cu_q, cu_k)
    dq, dk, dv = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k)
    torch.cuda.synchronize()
    assert not dq.any() and not dk.any() and dv.any()


def test_attention_scores_far_apart(cuda_device):
    """Scores in the thousands and one dominating key: no overflow, the maximum moves from tile to tile."""
    dev = cuda_device
    q, k, v, do, cu_q, cu_k = _inputs([90], [700], 2, 2, 64, "bf16", dev, seed=3)
    q = (q * 40).contiguous()
    k[650] = q[5, 0] / 8
    for causal in (False, True):
        o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=causal, scale=1.0)
        torch.cuda.synchronize()
        want, want_lse = stage.attention(_np(q), _np(k), _np(v), [0, 90], [0, 700], causal=causal, scale=1.0)
        # the scores reach 1e4 in fp32: an absolute error of 1e4 * 2^-22 in the exponent
        assert np.isfinite(_np(o)).all()
        assert np.abs(_np(lse) - want_lse).max() <= 1e-2
        assert np.linalg.norm(_np(o) - want) <= 1e-2 * np.linalg.norm(want)


def test_attention_nan_stays_in_its_sequence(cuda_device):
    dev, lens = cuda_device, [37, 70, 20]
    q, k, v, do, cu, _ = _inputs(lens, lens, 2, 1, 64, "bf16", dev, seed=4)
    o, lse = eq.attention(q, k, v, cu, cu)
    g = eq.attention_backward(do, q, k, v, o, lse, cu, cu)
    bad = [t.clone() for t in (q, k, v, do)]
    for t in bad:
        t[37:107] = float("nan")
    o2, lse2 = eq.attention(*bad[:3], cu, cu)
    g2 = eq.attention_backward(bad[3], *bad[:3], o2, lse2, cu, cu)
    torch.cuda.synchronize()
    keep = torch.ones(127, dtype=torch.bool)
    keep[37:107] = False
    for a, b in zip((o, lse, *g), (o2, lse2, *g2)):
        assert torch.equal(a[keep], b[keep]) and bool(b[~keep].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [([150], [150]), ([4], [700]), ([70, 33], [90, 33]), ([2, 3], [600, 900])],
                         ids=["prompt", "step", "longer", "steps"])
def test_attention_values_of_later_tokens(lens, dtype, cuda_device):
    """Infinities and NaN in tokens that a causal row must not see leave it alone, in o, lse and every gradient;
    the rows that see them get what the sums give."""
    dev, (lq, lk) = cuda_device, lens
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, 4, 2, 64, dtype, dev, seed=9)
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
    g = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=True)
    n_q, n_k = lq[0], lk[0]
    for late in (1, 2, n_q - 1):  # the last `late` tokens of the first sequence
        q2, k2, v2, do2 = (t.clone() for t in (q, k, v, do))
        v2[n_k - late, 0, 3] = float("inf")
        v2[n_k - late, 0, 5] = float("-inf")
        v2[n_k - late, 1, 7] = float("nan")
        o2, lse2 = eq.attention(q2, k2, v2, cu_q, cu_k, causal=True)
        torch.cuda.synchronize()
        keep = torch.ones(sum(lq), dtype=torch.bool)
        keep[n_q - late:n_q] = False
        assert torch.equal(lse, lse2) and torch.equal(o[keep], o2[keep])
        assert bool((o2[~keep][:, :2, 3] == float("inf")).all()) and bool((o2[~keep][:, :2, 5] == float("-inf")).all())
        assert bool(o2[~keep][:, 2:, 7].isnan().all())
        rest = [d for d in range(64) if d not in (3, 5, 7)]
        assert torch.equal(o2[:, :, rest], o[:, :, rest])
        k2[n_k - late:n_k] = float("nan")
        v2[n_k - late:n_k] = float("-inf")
        q2[n_q - late:n_q] = float("inf")
        do2[n_q - late:n_q] = float("nan")
        o2, lse2 = eq.attention(q2, k2, v2, cu_q, cu_k, causal=True)
        g2 = eq.attention_backward(do2, q2, k2, v2, o2, lse2, cu_q, cu_k, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
        assert bool(o2[~keep].isnan().all()) and bool(lse2[~keep].isnan().all())
        assert torch.equal(g[0][keep], g2[0][keep]) and bool(g2[0][~keep].isnan().all())
        # every key of the first sequence is seen by a row of NaN; the other sequences' are not
        for a, b in zip(g[1:], g2[1:]):
            assert bool(b[:n_k].isnan().all()) and torch.equal(a[n_k:], b[n_k:])
    # early rows of NaN reach only the keys they see
    do2, q2 = do.clone(), q.clone()
    do2[0], q2[0] = float("nan"), float("inf")
    o2, lse2 = eq.attention(q2, k, v, cu_q, cu_k, causal=True)
    g2 = eq.attention_backward(do2, q2, k, v, o2, lse2, cu_q, cu_k, causal=True)
    torch.cuda.synchronize()
    sees = n_k - n_q + 1
    for a, b in zip(g[1:], g2[1:]):
        assert bool(b[:sees].isnan().all()) and torch.equal(a[sees:], b[sees:])
    assert torch.equal(g[0][1:], g2[0][1:])
    do2 = do.clone()
    do2[0, 0, 11] = float("inf")  # one value: dv's column, and dk through delta
    g2 = eq.attention_backward(do2, q, k, v, o, lse, cu_q, cu_k, causal=True)
    torch.cuda.synchronize()
    assert bool((g2[2][:sees, 0, 11] == float("inf")).all()) and torch.equal(g2[2][sees:], g[2][sees:])
    assert torch.equal(g2[1][sees:], g[1][sees:]) and bool(torch.isfinite(g2[2][:sees, 0, :11]).all())


def test_attention_streams_and_repeats(cuda_device):
    """The same bits every time, on another stream than the tensors' own, and with the caller's workspace."""
    dev = cuda_device
    q, k, v, do, cu_q, cu_k = _inputs([1, 3, 200], [900, 1200, 200], 4, 2, 128, "bf16", dev, seed=6)
    o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
    g = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.full((1 << 26,), 0xff, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        for _ in range(3):
            o2, lse2 = eq.attention(q, k, v, cu_q, cu_k, causal=True, workspace=ws)
            g2 = eq.attention_backward(do, q, k, v, o2, lse2, cu_q, cu_k, causal=True, workspace=ws)
            side.synchronize()
            for a, b in zip((o, lse, *g), (o2, lse2, *g2)):
                assert torch.equal(a, b)


def test_attention_bounds_outside_the_tensors(cuda_device):
    """Sequence bounds that no caller should give stay inside the tensors (the results mean nothing)."""
    dev = cuda_device
    q, k, v, do, _, _ = _inputs([50], [80], 2, 2, 32, "f32", dev, seed=7)
    for bounds in ([0, 1000, 50], [-5, 20, 2 ** 31 - 1], [40, 10, 45]):
        cu = torch.tensor(bounds, dtype=torch.int32, device=dev)
        n = torch.tensor([10 ** 9, -3], dtype=torch.int32, device=dev)
        o, lse = eq.attention(q, k, v, cu, cu, len_k=n)
        eq.attention_backward(do, q, k, v, torch.zeros_like(q), torch.zeros_like(lse), cu, cu, len_k=n)
        torch.cuda.synchronize()


def test_attention_refusals(cuda_device):
    dev = cuda_device
    q, k, v, do, cu_q, cu_k = _inputs([10], [12], 4, 2, 32, "bf16", dev)
    o, lse = eq.attention(q, k, v, cu_q, cu_k)
    bad = [
        (ValueError, lambda: eq.attention(q[:, :, :16], k, v, cu_q, cu_k)),
        (ValueError, lambda: eq.attention(q, k, v[:11], cu_q, cu_k)),
        (TypeError, lambda: eq.attention(q, k.half(), v, cu_q, cu_k)),
        (TypeError, lambda: eq.attention(q.cpu(), k, v, cu_q, cu_k)),
        (ValueError, lambda: eq.attention(q, k, v, cu_q.long(), cu_k)),
        (ValueError, lambda: eq.attention(q, k, v, cu_q, cu_k[:1])),
        (ValueError, lambda: eq.attention(q.transpose(1, 2), k, v, cu_q, cu_k)),
        (eq.EqlinError, lambda: eq.attention(q[:, :3], k, v, cu_q, cu_k)),          # 3 heads on 2
        (eq.EqlinError, lambda: eq.attention(q, k, v, cu_q, cu_k, scale=0.0)),
        (eq.EqlinError, lambda: eq.attention(q, k, v, cu_q, cu_k, scale=float("nan"))),
        (eq.EqlinError, lambda: eq.attention(q, k, v, cu_q, cu_k, out=q)),
        (ValueError, lambda: eq.attention_backward(do[:9], q, k, v, o, lse, cu_q, cu_k)),
        (ValueError, lambda: eq.attention_backward(do, q, k, v, o, lse.double(), cu_q, cu_k)),
        (eq.EqlinError, lambda: eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, dk=k)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    x = torch.zeros((4, 2, 136), dtype=torch.bfloat16, device=dev)
    cu = _cu([4], dev)
    for t in (x, x[:, :, :12], x[:, :, 4:36]):  # dim > 128; dim % 8; a pointer off 16 bytes
        with pytest.raises(eq.EqlinError):
            eq.attention(t, t, t, cu, cu)
    e = torch.zeros((0, 2, 32), dtype=torch.bfloat16, device=dev)
    o, lse = eq.attention(e, e, e, _cu([], dev), _cu([], dev))
    assert o.shape == (0, 2, 32) and lse.shape == (0, 2)
    o, lse = eq.attention(q, e, e, cu_q, torch.zeros_like(cu_q))  # no keys at all
    dq, dk, dv = eq.attention_backward(do[:, :4], q, e, e, o, lse, cu_q, torch.zeros_like(cu_q))
    torch.cuda.synchronize()
    assert not o.any() and bool(lse.isneginf().all()) and not dq.any()
