"""The transformer-stage operators around the EQ-Linear layers, as measured cases.

A stage of an equivariant transformer holds its tokens as x[N, C, G] (group axis innermost) and runs
norm -> EQ-Linear (q, k, v) -> rotary positions -> attention -> EQ-Linear -> norm with the residual -> MLP
block. The cases time the three operators between the layers, each direction and type, from one token to the
long sequences:

* ``norm*``: root-mean-square norm over a token's C * G values with the residual's addition (``norm``),
  the same with an 8-bit (e4m3) output and one scale a token (``norm_quant``), forward plus gradients
  (``norm_train``);
* ``rotary*``: rotary positions over 1 to 3 axes, the last two turned by the inverse of each group element
  (``rotary``), rotation plus the gradient's inverse rotation (``rotary_train``);
* ``attn*``: attention over packed sequences with grouped heads, causal or full (``attn``; with one query
  a sequence it is the step over a cache), forward plus gradients (``attn_train``).

A case's ``run`` is the plain form in fp32 torch operations, or, where ``own`` is set, the calls of
``fourier_domain_linear_amd`` that a user makes.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0
E4M3_MAX = 448.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELEM = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one new token in each of 8 streams, p4 stage of 192 channels: the latency of the smallest norm
        {"name": "norm_n8_c192g4_f32", "op": "norm", "N": 8, "C": 192, "G": 4, "dtype": "f32"},
        # the p8 stage of 64 images of 14 x 14 tokens, 256 channels, normalised into an 8-bit operand
        {"name": "norm_quant_n12544_c256g8_f16", "op": "norm_quant", "N": 12544, "C": 256, "G": 8, "dtype": "f16"},
        # a training step's norm at the p4 stage of 8 images of 56 x 56 tokens, 96 channels
        {"name": "norm_train_n25088_c96g4_bf16", "op": "norm_train", "N": 25088, "C": 96, "G": 4, "dtype": "bf16"},
        # one new token of 64 video streams, plain heads of 128 (no group axis), time / height / width
        {"name": "rotary_n64_h18_d128_bf16", "op": "rotary", "N": 64, "H": 18, "dc": 128, "G": 1, "axes": 3,
         "dtype": "bf16"},
        # q and k of the p8 stage (64 x 14 x 14 tokens, 16 + 16 heads of 16 channels x 8), with gradients
        {"name": "rotary_train_n12544_h32_d16g8_bf16", "op": "rotary_train", "N": 12544, "H": 32, "dc": 16, "G": 8,
         "axes": 2, "dtype": "bf16"},
        # the smallest call: one 8 x 8 image, p4 with 16 channels as two heads of 8 channels x 4, fp32
        {"name": "attn_1x64_h2_d32_f32", "op": "attn", "B": 1, "lq": 64, "lk": 64, "Hq": 2, "Hkv": 2, "D": 32,
         "causal": False, "ragged": 0, "dtype": "f32"},
        # one new token in each of 8 streams over caches of up to 32768, 16 query heads on 2 key-value heads
        {"name": "attn_8x1_over_32768_h16kv2_d128_bf16", "op": "attn", "B": 8, "lq": 1, "lk": 32768, "Hq": 16,
         "Hkv": 2, "D": 128, "causal": True, "ragged": 3, "dtype": "bf16"},
        # the p8 stage: 64 images of 14 x 14 tokens, 256 channels x 8 as 16 heads of 128
        {"name": "attn_64x196_h16_d128_bf16", "op": "attn", "B": 64, "lq": 196, "lk": 196, "Hq": 16, "Hkv": 16,
         "D": 128, "causal": False, "ragged": 0, "dtype": "bf16"},
        # 24 images of different sizes packed together, up to 56 x 56 tokens, p4 with 96 channels as 6 heads of 64
        {"name": "attn_24ragged3136_h6_d64_f16", "op": "attn", "B": 24, "lq": 3136, "lk": 3136, "Hq": 6, "Hkv": 6,
         "D": 64, "causal": False, "ragged": 5, "dtype": "f16"},
        # two long prompts, causal, 16 query heads on 4 key-value heads
        {"name": "attn_2x8192_causal_h16kv4_d128_bf16", "op": "attn", "B": 2, "lq": 8192, "lk": 8192, "Hq": 16,
         "Hkv": 4, "D": 128, "causal": True, "ragged": 0, "dtype": "bf16"},
        # a training step at the p4 stage: 16 images of 28 x 28 tokens, 192 channels x 4 as 12 heads of 64
        {"name": "attn_train_16x784_h12_d64_bf16", "op": "attn_train", "B": 16, "lq": 784, "lk": 784, "Hq": 12,
         "Hkv": 12, "D": 64, "causal": False, "ragged": 0, "dtype": "bf16"},
        # a training step on packed causal sequences of up to 4096 tokens, grouped heads of 128
        {"name": "attn_train_4ragged4096_causal_h16kv4_d128_bf16", "op": "attn_train", "B": 4, "lq": 4096,
         "lk": 4096, "Hq": 16, "Hkv": 4, "D": 128, "causal": True, "ragged": 2, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_quant", "norm_train", "rotary", "rotary_train", "attn", "attn", "attn", "attn_train",
                     "attn_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("norm"):
        G = rng.choice([1, 2, 4, 8])
        C = _log(rng, 16, 2048 // G) if rng.random() < 0.3 else 8 * _log(rng, 2, 256 // G)
        return {"op": op, "N": _log(rng, 1, 25088), "C": C, "G": G, "dtype": dtype}
    if op.startswith("rotary"):
        G = rng.choice([1, 2, 4, 8])
        return {"op": op, "N": _log(rng, 1, 12544), "H": _log(rng, 1, 32), "dc": rng.choice([64, 96, 128]) // G, "G": G,
                "axes": rng.choice([1, 2, 3]), "dtype": dtype}
    Hkv = _log(rng, 1, 8)
    Hq = Hkv * rng.choice([n for n in (1, 1, 2, 4) if n * Hkv <= 16])
    D = rng.choice([32, 40, 64, 64, 96, 128, 128])
    causal = rng.random() < 0.5
    if op == "attn" and rng.random() < 0.35:  # one or a few new tokens over a cache
        lk = _log(rng, 64, 32768)
        B = _log(rng, 1, max(1, min(64, 8 * 32768 // lk)))
        lq = min(rng.choice([1, 1, 1, 4]), lk)
    else:  # prompts, images
        lk = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 2 ** (28 if op == "attn" else 27) // (lk * lk * Hq))))
        lq = lk
    return {"op": op, "B": B, "lq": lq, "lk": lk, "Hq": Hq, "Hkv": Hkv, "D": D, "causal": causal,
            "ragged": rng.randrange(100) if B > 1 else 0, "dtype": dtype}


def _lengths(case):
    """(query lengths, key lengths) of the packed sequences. ``ragged`` seeds lengths spread between an
    eighth of the longest and the longest; a cache step keeps its few queries."""
    B, lq, lk = case["B"], case["lq"], case["lk"]
    if not case["ragged"]:
        return [lq] * B, [lk] * B
    rng = random.Random(case["ragged"])
    ks = [lk] + [min(lk, max(lq if lq < lk else 1, _log(rng, max(1, lk // 8), lk))) for _ in range(B - 1)]
    return (ks if lq == lk else [lq] * B), ks


def _pairs(case):
    """Channel pairs for each axis: all of them, the later axes taking the remainder."""
    P, A = case["dc"] // 2, case["axes"]
    return [P // A] * (A - 1) + [P - P // A * (A - 1)]


def _positions(case):
    """Token positions [N, axes]: (time, row, column) of 14 x 14 images one after the other."""
    n = torch.arange(case["N"])
    cols = [n // 196 % 512, n % 196 // 14, n % 14]
    return torch.stack(cols[3 - case["axes"]:], 1).to(torch.int32)


def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    st = dict(case)
    if case["op"].startswith("norm"):
        shape = (case["N"], case["C"], case["G"])
        st["x"] = _randn(shape, gen, dt)
        st["residual"] = _randn(shape, gen, dt)
        st["gamma"] = (1 + 0.1 * torch.randn(case["C"], generator=gen, device="cuda")).to(dt)
        if case["op"] == "norm_train":
            st["dy"] = _randn(shape, gen, dt)
            st["ds"] = _randn(shape, gen, dt)
    elif case["op"].startswith("rotary"):
        shape = (case["N"], case["H"], case["dc"], case["G"])
        st["x"] = _randn(shape, gen, dt)
        st["pos"] = _positions(case).cuda()
        st["pairs"] = _pairs(case)
        if case["op"] == "rotary_train":
            st["dy"] = _randn(shape, gen, dt)
    else:
        qs, ks = _lengths(case)
        cu = lambda v: torch.tensor([0] + v, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
        st["cu_q"], st["cu_k"] = cu(qs), cu(ks)
        st["max_q"], st["max_k"] = max(qs), max(ks)
        st["q"] = _randn((sum(qs), case["Hq"], case["D"]), gen, dt)
        st["k"] = _randn((sum(ks), case["Hkv"], case["D"]), gen, dt)
        st["v"] = _randn((sum(ks), case["Hkv"], case["D"]), gen, dt)
        if case["op"] == "attn_train":
            st["do"] = _randn((sum(qs), case["Hq"], case["D"]), gen, dt)
    return st


# ---- the plain forms ----


def _norm(st):
    s = st["x"].float() + st["residual"].float()
    rstd = torch.rsqrt((s * s).mean(dim=(1, 2)) + EPS)
    y = s * rstd[:, None, None] * st["gamma"].float()[None, :, None]
    return s, rstd, y


def _norm_plain(st):
    dt = st["x"].dtype
    s, rstd, y = _norm(st)
    if st["op"] == "norm":
        return y.to(dt), s.to(dt), rstd
    if st["op"] == "norm_quant":
        scale = y.abs().amax(dim=(1, 2)) / E4M3_MAX
        q = (y / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return q, scale, s.to(dt), rstd
    # the gradients see the sum as the forward stored it
    dy, sf = st["dy"].float(), s.to(dt).float()
    xh = sf * rstd[:, None, None]
    w = dy * st["gamma"].float()[None, :, None]
    dx = st["ds"].float() + rstd[:, None, None] * (w - xh * (w * xh).mean(dim=(1, 2), keepdim=True))
    return y.to(dt), s.to(dt), dx.to(dt), (dy * xh).sum(dim=(0, 2))


def _turned(pos, G):
    """The positions that group element g sees: [N, G, axes], the last two axes turned by -360 g / G degrees."""
    p = pos.float()[:, None, :].expand(-1, G, -1)
    if p.shape[2] < 2 or G == 1:
        return p
    t = torch.arange(G, device=pos.device) * (2 * math.pi / G)
    c, s = torch.cos(t), torch.sin(t)
    row, col = p[..., -2], p[..., -1]
    return torch.cat([p[..., :-2], (row * c + col * s)[..., None], (col * c - row * s)[..., None]], 2)


def _rotate(x, pos, pairs, sign):
    n, G, P = len(pairs), x.shape[3], sum(pairs)
    axis = torch.arange(n, device=x.device).repeat_interleave(torch.tensor(pairs, device=x.device), output_size=P)
    width = torch.tensor(pairs, device=x.device, dtype=torch.float32)
    first = torch.cumsum(width, 0) - width
    freq = torch.exp(-math.log(BASE) * (torch.arange(P, device=x.device) - first[axis]) / width[axis])
    ang = _turned(pos, G)[:, :, axis] * freq  # [N, G, P]
    c, s = torch.cos(ang).transpose(1, 2)[:, None], sign * torch.sin(ang).transpose(1, 2)[:, None]
    a, b, rest = x[:, :, :P].float(), x[:, :, P:2 * P].float(), x[:, :, 2 * P:].float()
    return torch.cat([a * c - b * s, a * s + b * c, rest], 2).to(x.dtype)


def _rotary_plain(st):
    y = _rotate(st["x"], st["pos"], st["pairs"], 1.0)
    return y if st["op"] == "rotary" else (y, _rotate(st["dy"], st["pos"], st["pairs"], -1.0))


def _rows(cu, total):
    """(sequence, place in it) of every packed token."""
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, t - cu[b]


def _padded(x, cu, longest, heads):
    """Packed [T, H, D] -> fp32 [B * heads, (H / heads) * longest, D], and which places hold a token."""
    at = torch.arange(longest, device=x.device)
    ok = at < (cu[1:] - cu[:-1])[:, None]
    i = (cu[:-1, None] + at).clamp(max=x.shape[0] - 1)
    y = x.float()[i] * ok[:, :, None, None]
    B, H, D = ok.shape[0], x.shape[1], x.shape[2]
    return y.view(B, longest, heads, H // heads, D).permute(0, 2, 3, 1, 4).reshape(B * heads, -1, D), ok


def _packed(y, cu, total, heads, longest):
    """The inverse of _padded."""
    b, i = _rows(cu, total)
    D = y.shape[-1]
    return y.view(cu.shape[0] - 1, heads, -1, longest, D)[b, :, :, i].reshape(total, -1, D)


def _attn_plain(st):
    q, k, v, cu_q, cu_k, Lq, Lk = (st[n] for n in ("q", "k", "v", "cu_q", "cu_k", "max_q", "max_k"))
    Hkv, dt, scale = k.shape[1], q.dtype, q.shape[2] ** -0.5
    qp, okq = _padded(q, cu_q, Lq, Hkv)
    kp, okk = _padded(k, cu_k, Lk, Hkv)
    vp, _ = _padded(v, cu_k, Lk, Hkv)
    B = okq.shape[0]
    ok = okq[:, :, None] & okk[:, None, :]
    if st["causal"]:
        shift = (cu_k[1:] - cu_k[:-1]) - (cu_q[1:] - cu_q[:-1])
        ok = ok & (torch.arange(Lk, device=q.device)[None, None, :]
                   <= torch.arange(Lq, device=q.device)[None, :, None] + shift[:, None, None])
    s = torch.bmm(qp, kp.transpose(1, 2)).mul_(scale).view(B, Hkv, -1, Lq, Lk)
    s = s.masked_fill_(~ok[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    lse = _packed((m + torch.log(total)).view(B * Hkv, -1, 1), cu_q, q.shape[0], Hkv, Lq)[:, :, 0]
    p = p.div_(total.clamp(min=torch.finfo(torch.float32).tiny)).view(B * Hkv, -1, Lk)
    o = _packed(torch.bmm(p, vp), cu_q, q.shape[0], Hkv, Lq).to(dt)
    if st["op"] == "attn":
        return o, lse
    dop, _ = _padded(st["do"], cu_q, Lq, Hkv)
    dv = torch.bmm(p.transpose(1, 2), dop)
    dp = torch.bmm(dop, vp.transpose(1, 2))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = torch.bmm(ds, kp), torch.bmm(ds.transpose(1, 2), qp)
    return (o, _packed(dq, cu_q, q.shape[0], Hkv, Lq).to(dt), _packed(dk, cu_k, k.shape[0], Hkv, Lk).to(dt),
            _packed(dv, cu_k, k.shape[0], Hkv, Lk).to(dt))


# ---- the framework's operators ----


def _run_own(st):
    import fourier_domain_linear_amd as eq

    op = st["op"]
    if op == "norm":
        return eq.rmsnorm(st["x"], st["gamma"], residual=st["residual"], eps=EPS)
    if op == "norm_quant":
        return eq.rmsnorm_quant(st["x"], st["gamma"], residual=st["residual"], eps=EPS)
    if op == "norm_train":
        y, s, rstd = eq.rmsnorm(st["x"], st["gamma"], residual=st["residual"], eps=EPS)
        dx, dgamma = eq.rmsnorm_backward(st["dy"], s, st["gamma"], rstd, ds=st["ds"])
        return y, s, dx, dgamma
    if op == "rotary":
        return eq.rotary(st["x"], st["pos"], st["pairs"], base=BASE)
    if op == "rotary_train":
        return (eq.rotary(st["x"], st["pos"], st["pairs"], base=BASE),
                eq.rotary(st["dy"], st["pos"], st["pairs"], base=BASE, inverse=True))
    o, lse = eq.attention(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], causal=st["causal"])
    if op == "attn":
        return o, lse
    return (o, *eq.attention_backward(st["do"], st["q"], st["k"], st["v"], o, lse, st["cu_q"], st["cu_k"],
                                      causal=st["causal"]))


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    return _norm_plain(state) if op.startswith("norm") else _rotary_plain(state) if op.startswith("rotary") \
        else _attn_plain(state)


def work(case):
    e, op = ELEM[case["dtype"]], case["op"]
    if op.startswith("norm"):
        n = case["N"] * case["C"] * case["G"]
        if op == "norm":
            return {"bytes": n * 4 * e + 4 * case["N"], "flops": 5 * n}
        if op == "norm_quant":
            return {"bytes": n * (3 * e + 1) + 8 * case["N"], "flops": 8 * n}
        return {"bytes": n * 7 * e + 4 * case["N"], "flops": 16 * n}
    if op.startswith("rotary"):
        n, times = case["N"] * case["H"] * case["dc"] * case["G"], 2 if op == "rotary_train" else 1
        return {"bytes": times * (2 * n * e + 4 * case["N"] * case["axes"]), "flops": times * 3 * n}
    qs, ks = _lengths(case)
    seen = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(qs, ks))
    q, k = sum(qs) * case["Hq"] * case["D"], sum(ks) * case["Hkv"] * case["D"]
    if op == "attn":
        return {"bytes": e * (2 * q + 2 * k) + 4 * sum(qs) * case["Hq"], "flops": 4 * seen * case["Hq"] * case["D"]}
    return {"bytes": e * (4 * q + 4 * k), "flops": 14 * seen * case["Hq"] * case["D"]}


# ---- the definitions in 64 bits ----


def _exact_norm(st):
    x, r, g = st["x"].double(), st["residual"].double(), st["gamma"].double().view(1, -1, 1)
    s = x + r
    if st["op"] == "norm_train":
        # gradients at the stored sum, by automatic differentiation; the forward at the exact one
        v = s.to(st["x"].dtype).double().flatten(1).requires_grad_(True)
        gam = st["gamma"].double().requires_grad_(True)
        rstd = (s.flatten(1).pow(2).sum(1) / v.shape[1] + EPS).pow(-0.5)
        out = v * (v.pow(2).mean(1, keepdim=True) + EPS).pow(-0.5) * gam.repeat_interleave(s.shape[2])[None]
        dv, dg = torch.autograd.grad(out, (v, gam), st["dy"].double().flatten(1))
        return (s * rstd[:, None, None] * g, s, (dv + st["ds"].double().flatten(1)).view(s.shape), dg)
    rstd = (s.flatten(1).pow(2).sum(1) / (s.shape[1] * s.shape[2]) + EPS).pow(-0.5)
    y = torch.einsum("n,ncg->ncg", rstd, s) * g
    if st["op"] == "norm":
        return y, s, rstd
    scale = y.flatten(1).abs().max(1).values / E4M3_MAX
    return y / scale.view(-1, 1, 1), scale, s, rstd


def _exact_rotary(st):
    def one(x, sign):
        x, out, j = x.double(), x.double().clone(), 0
        P, G = sum(st["pairs"]), x.shape[3]
        for axis, count in enumerate(st["pairs"]):
            back = len(st["pairs"]) - axis  # 2: rows, 1: columns, 3: time
            for i in range(count):
                for h in range(G):
                    p = st["pos"][:, axis].double()
                    if len(st["pairs"]) > 1 and back <= 2:
                        t = 2 * math.pi * h / G
                        row, col = st["pos"][:, -2].double(), st["pos"][:, -1].double()
                        p = row * math.cos(t) + col * math.sin(t) if back == 2 else col * math.cos(t) - row * math.sin(t)
                    z = torch.polar(torch.ones_like(p), sign * p * BASE ** (-i / count))[:, None]
                    z = torch.complex(x[:, :, j, h], x[:, :, j + P, h]) * z
                    out[:, :, j, h], out[:, :, j + P, h] = z.real, z.imag
                j += 1
        return out

    return one(st["x"], 1) if st["op"] == "rotary" else (one(st["x"], 1), one(st["dy"], -1))


def _exact_attn(st):
    train = st["op"] == "attn_train"
    q, k, v = (st[n].double() for n in "qkv")
    outs = [torch.zeros_like(q), torch.zeros(q.shape[:2], device=q.device, dtype=q.dtype)] + \
        ([torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)] if train else [])
    qe, ke, grp = st["cu_q"].tolist(), st["cu_k"].tolist(), q.shape[1] // k.shape[1]
    for b in range(len(qe) - 1):
        rq, rk = slice(qe[b], qe[b + 1]), slice(ke[b], ke[b + 1])
        nq, nk = qe[b + 1] - qe[b], ke[b + 1] - ke[b]
        hide = torch.ones(nq, nk, dtype=torch.bool, device=q.device).triu(nk - nq + 1) if st["causal"] else None
        for h in range(q.shape[1]):
            qh, kh, vh = (t.detach().contiguous().requires_grad_(train) for t in
                          (q[rq, h], k[rk, h // grp], v[rk, h // grp]))
            s = qh @ kh.T / math.sqrt(q.shape[2])
            s = s if hide is None else s.masked_fill(hide, -math.inf)
            o = torch.softmax(s, 1) @ vh
            outs[0][rq, h], outs[1][rq, h] = o.detach(), torch.logsumexp(s.detach(), 1)
            if train:
                dq, dk, dv = torch.autograd.grad(o, (qh, kh, vh), st["do"][rq, h].double())
                outs[2][rq, h] = dq
                outs[3][rk, h // grp] += dk
                outs[4][rk, h // grp] += dv
    return tuple(outs[:2]) if not train else (outs[0], *outs[2:])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    return _exact_norm(st) if op.startswith("norm") else _exact_rotary(st) if op.startswith("rotary") \
        else _exact_attn(st)
