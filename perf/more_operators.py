"""The recurrent stage's operators beside the EQ-Linear layers, as measured cases.

A recurrent stage holds its tokens as x[N, C, G] (group axis innermost) and runs layer norm -> EQ-Linear (values, forget gates,
output gates) -> gated recurrence over each sequence's tokens -> EQ-Linear -> layer norm with the residual. The cases time
the two operators, each direction and type, from one token to the long sequences:

* ``ln*``: layer norm over a token's C * G values with the residual's addition (``ln``), forward plus gradients (``ln_train``);
* ``rec*``: the gated linear recurrence h = f h + (1 - f) x, f = sigmoid(forget), over packed sequences, with an output gate
  and initial states or without (``rec``; with one token a sequence it is the serving step), forward plus gradients (``rec_train``).

A case's ``run`` is the plain form in fp32 torch operations, or, where ``own`` is set, the calls of
``fourier_domain_linear_amd`` that a user makes.
"""
import math
import random

import torch

own = False

EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELEM = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one new token in each of 8 streams, p4 stage of 192 channels: the latency of the smallest norm
        {"name": "ln_n8_c192g4_f32", "op": "ln", "N": 8, "C": 192, "G": 4, "dtype": "f32"},
        # the p8 stage of 64 images of 14 x 14 tokens, 256 channels
        {"name": "ln_n12544_c256g8_bf16", "op": "ln", "N": 12544, "C": 256, "G": 8, "dtype": "bf16"},
        # a training step's norm at the p4 stage of 8 images of 56 x 56 tokens, 96 channels
        {"name": "ln_train_n25088_c96g4_bf16", "op": "ln_train", "N": 25088, "C": 96, "G": 4, "dtype": "bf16"},
        # rows of an odd length without a group axis, in fp32: no whole number of vectors
        {"name": "ln_train_n12543_c181g1_f32", "op": "ln_train", "N": 12543, "C": 181, "G": 1, "dtype": "f32"},
        # one new token in each of 8 streams: the latency of the smallest step, states in and out
        {"name": "rec_8x1_c192g4_bf16", "op": "rec", "B": 8, "len": 1, "C": 192, "G": 4, "ragged": 0, "gate": True,
         "state": True, "reverse": False, "dtype": "bf16"},
        # the same for many streams of the p8 stage of 64 channels, in fp32
        {"name": "rec_1024x1_c64g8_f32", "op": "rec", "B": 1024, "len": 1, "C": 64, "G": 8, "ragged": 0, "gate": False,
         "state": True, "reverse": False, "dtype": "f32"},
        # the p8 stage: 64 images of 14 x 14 tokens, 256 channels x 8, with the output gate
        {"name": "rec_64x196_c256g8_bf16", "op": "rec", "B": 64, "len": 196, "C": 256, "G": 8, "ragged": 0, "gate": True,
         "state": False, "reverse": False, "dtype": "bf16"},
        # 24 images of different sizes packed together, up to 56 x 56 tokens, p4 with 96 channels, last token first
        {"name": "rec_24ragged3136_c96g4_f16", "op": "rec", "B": 24, "len": 3136, "C": 96, "G": 4, "ragged": 5, "gate": False,
         "state": False, "reverse": True, "dtype": "f16"},
        # one long stream of the same stage
        {"name": "rec_1x65536_c96g4_bf16", "op": "rec", "B": 1, "len": 65536, "C": 96, "G": 4, "ragged": 0, "gate": False,
         "state": True, "reverse": False, "dtype": "bf16"},
        # a training step at the p4 stage: 16 images of 28 x 28 tokens, 192 channels x 4, with the output gate
        {"name": "rec_train_16x784_c192g4_bf16", "op": "rec_train", "B": 16, "len": 784, "C": 192, "G": 4, "ragged": 0,
         "gate": True, "state": False, "reverse": False, "dtype": "bf16"},
        # a training step on packed sequences of up to 4096 tokens at the p8 stage, states handed from piece to piece
        {"name": "rec_train_4ragged4096_c256g8_bf16", "op": "rec_train", "B": 4, "len": 4096, "C": 256, "G": 8, "ragged": 2,
         "gate": False, "state": True, "reverse": False, "dtype": "bf16"},
        # the same on ragged sequences of odd lengths and an odd width, fp32, last token first
        {"name": "rec_train_7ragged1001_c99g1_f32", "op": "rec_train", "B": 7, "len": 1001, "C": 99, "G": 1, "ragged": 3,
         "gate": True, "state": True, "reverse": True, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_train", "ln_train", "rec", "rec", "rec", "rec_train", "rec_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    G = rng.choice([1, 2, 4, 8])
    if op.startswith("ln"):
        C = _log(rng, 16, 2048 // G) if rng.random() < 0.3 else 8 * _log(rng, 2, 256 // G)
        return {"op": op, "N": _log(rng, 1, 25088), "C": C, "G": G, "dtype": dtype}
    C = _log(rng, 9, 2048 // G) if rng.random() < 0.3 else 8 * _log(rng, 2, 256 // G)
    most = (24 if op == "rec" else 23) - (1 if dtype == "f32" else 0)  # log2 of the values a tensor
    length = 1 if op == "rec" and rng.random() < 0.3 else _log(rng, 2, min(65536 if op == "rec" else 8192, 2 ** most // (C * G)))
    B = _log(rng, 1, max(1, min(1024, 2 ** most // (C * G * length))))
    return {"op": op, "B": B, "len": length, "C": C, "G": G, "ragged": rng.randrange(100) if B > 1 and length > 1 else 0,
            "gate": rng.random() < 0.5, "state": length == 1 or rng.random() < 0.5, "reverse": rng.random() < 0.3, "dtype": dtype}


def _lengths(case):
    """Tokens of each packed sequence. ``ragged`` seeds lengths spread between an eighth of the longest and the longest."""
    B, n = case["B"], case["len"]
    if not case["ragged"]:
        return [n] * B
    rng = random.Random(case["ragged"])
    return [n] + [min(n, _log(rng, max(1, n // 8), n)) for _ in range(B - 1)]


def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, C, G = DTYPES[case["dtype"]], case["C"], case["G"]
    st = dict(case)
    if case["op"].startswith("ln"):
        shape = (case["N"], C, G)
        # a stream with a common part, as residual streams have
        st["x"] = _randn(shape, gen, dt)
        st["residual"] = (_randn(shape, gen, torch.float32) + 0.5).to(dt)
        st["gamma"] = (1 + 0.1 * torch.randn(C, generator=gen, device="cuda")).to(dt)
        st["beta"] = (0.1 * torch.randn(C, generator=gen, device="cuda")).to(dt)
        if case["op"] == "ln_train":
            st["dy"] = _randn(shape, gen, dt)
            st["ds"] = _randn(shape, gen, dt)
        return st
    lens = _lengths(case)
    T, B = sum(lens), len(lens)
    # one layer's output, its channels dealt to values, forget gates and output gates: the operands are strided parts of
    # it. Channels forget at rates from half a token to hundreds of tokens.
    parts = 3 if case["gate"] else 2
    packed = _randn((T, parts * C, G), gen, torch.float32)
    packed[:, C:2 * C] += torch.linspace(-1, 6, C, device="cuda")[None, :, None]
    st["packed"] = packed.to(dt)
    st["x"], st["forget"] = st["packed"][:, :C], st["packed"][:, C:2 * C]
    st["out_gate"] = st["packed"][:, 2 * C:] if case["gate"] else None
    st["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    st["longest"] = max(lens)
    st["h0"] = _randn((B, C, G), gen, torch.float32) if case["state"] else None
    if case["op"] == "rec_train":
        st["dy"] = _randn((T, C, G), gen, dt)
        st["dfinal"] = _randn((B, C, G), gen, torch.float32) if case["state"] else None
    return st


# ---- the plain forms ----


def _ln_plain(st):
    dt = st["x"].dtype
    s = st["x"].float() + st["residual"].float()
    mean = s.mean(dim=(1, 2))
    d = s - mean[:, None, None]
    rstd = torch.rsqrt((d * d).mean(dim=(1, 2)) + EPS)
    gamma = st["gamma"].float()[None, :, None]
    y = d * rstd[:, None, None] * gamma + st["beta"].float()[None, :, None]
    if st["op"] == "ln":
        return y.to(dt), s.to(dt), mean, rstd
    # the gradients see the sum as the forward stored it
    dy = st["dy"].float()
    xh = (s.to(dt).float() - mean[:, None, None]) * rstd[:, None, None]
    w = dy * gamma
    dx = w - w.mean(dim=(1, 2), keepdim=True) - xh * (w * xh).mean(dim=(1, 2), keepdim=True)
    dx = st["ds"].float() + rstd[:, None, None] * dx
    return y.to(dt), s.to(dt), dx.to(dt), (dy * xh).sum(dim=(0, 2)), dy.sum(dim=(0, 2))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling."""
    d, n = 1, a.shape[1]
    while d < n:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _rec_plain(st):
    cu, dt, C, G = st["cu"].long(), st["x"].dtype, st["C"], st["G"]
    n, T = st["longest"], st["x"].shape[0]
    at = torch.arange(n, device=cu.device)[None, :]
    lens = (cu[1:] - cu[:-1])[:, None]
    ok = (at < lens)[:, :, None]
    rows = (cu[1:, None] - 1 - at if st["reverse"] else cu[:-1, None] + at).clamp(0, T - 1)
    pad = lambda t: t.reshape(T, C * G).float()[rows]  # noqa: E731
    flat = rows[ok[:, :, 0]]

    def packed(t):  # back to [T, C, G]
        out = torch.empty((T, C * G), dtype=dt, device=t.device)
        out[flat] = t[ok[:, :, 0]].to(dt)
        return out.view(T, C, G)

    x, z = pad(st["x"]), pad(st["forget"])
    f = torch.where(ok, torch.sigmoid(z), torch.ones_like(z))  # past the end: the state stays
    keep = torch.where(ok, torch.sigmoid(-z), torch.zeros_like(z))
    h0 = torch.zeros_like(x[:, 0]) if st["h0"] is None else st["h0"].view(-1, C * G)
    b = keep * x
    b = torch.cat([b[:, :1] + f[:, :1] * h0[:, None], b[:, 1:]], 1)
    h = _scan(f, b)
    o = pad(st["out_gate"]) if st["gate"] else None
    y = h * (o * torch.sigmoid(o)) if st["gate"] else h
    final = h[:, -1].view(-1, C, G)
    if st["op"] == "rec":
        return packed(y), final
    dy = pad(st["dy"]) * ok
    direct = dy * (o * torch.sigmoid(o)) if st["gate"] else dy
    dlast = torch.zeros_like(h0) if st["dfinal"] is None else st["dfinal"].view(-1, C * G)
    direct = torch.cat([direct[:, :-1], direct[:, -1:] + dlast[:, None]], 1)
    after = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)
    dh = _scan(after.flip(1), direct.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    grads = [packed(keep * dh), packed(dh * (before - x) * f * keep)]
    if st["gate"]:
        sig = torch.sigmoid(o)
        grads.append(packed(dy * h * sig * (1 + o * (1 - sig))))
    outs = [packed(y), final, torch.cat(grads, 1)]
    return tuple(outs + ([(f[:, 0] * dh[:, 0]).view(-1, C, G)] if st["state"] else []))


# ---- the framework's operators ----


def _run_own(st):
    import fourier_domain_linear_amd as eq

    op = st["op"]
    if op.startswith("ln"):
        y, s, mean, rstd = eq.layernorm(st["x"], st["gamma"], st["beta"], residual=st["residual"], eps=EPS)
        if op == "ln":
            return y, s, mean, rstd
        return (y, s, *eq.layernorm_backward(st["dy"], s, st["gamma"], mean, rstd, ds=st["ds"]))
    how = {"gate": st["out_gate"], "reverse": st["reverse"], "longest": st["longest"]}
    y, final, marks = eq.recurrence(st["x"], st["forget"], st["cu"], state=st["h0"], with_marks=op == "rec_train", **how)
    if op == "rec":
        return y, final
    C = st["C"]
    grad = torch.empty_like(st["packed"])  # the gradient of the layer's output, in its parts
    _, _, _, dstate = eq.recurrence_backward(st["dy"], st["x"], st["forget"], st["cu"], marks, dfinal=st["dfinal"],
                                             with_state=st["state"], dx=grad[:, :C], dforget=grad[:, C:2 * C],
                                             dgate=grad[:, 2 * C:] if st["gate"] else None, **how)
    return (y, final, grad, dstate) if st["state"] else (y, final, grad)


def run(state):
    if own:
        return _run_own(state)
    return _ln_plain(state) if state["op"].startswith("ln") else _rec_plain(state)


def work(case):
    e, op, L = ELEM[case["dtype"]], case["op"], case["C"] * case["G"]
    if op.startswith("ln"):
        n = case["N"] * L
        if op == "ln":
            return {"bytes": n * 4 * e + 8 * case["N"], "flops": 8 * n}
        return {"bytes": n * 7 * e, "flops": 20 * n}
    n, states = sum(_lengths(case)) * L, 4 * case["B"] * L
    gate, state = int(case["gate"]), int(case["state"])
    if op == "rec":
        return {"bytes": n * e * (3 + gate) + states * (1 + state), "flops": n * (8 + 6 * gate)}
    return {"bytes": n * e * (6 + 2 * gate) + states * (1 + 2 * state), "flops": n * (22 + 18 * gate)}


# ---- the definitions in 64 bits ----


def _exact_ln(st):
    x, r = st["x"].double(), st["residual"].double()
    s = x + r
    eps, n = EPS, s.shape[1] * s.shape[2]
    mean = torch.einsum("ncg->n", s) / n
    var = torch.einsum("ncg,ncg->n", s, s) / n - mean ** 2
    rstd = 1 / torch.sqrt(var + eps)
    y = torch.einsum("ncg,n,c->ncg", s - mean.view(-1, 1, 1), rstd, st["gamma"].double()) + st["beta"].double().view(1, -1, 1)
    if st["op"] == "ln":
        return y, s, mean, rstd
    # the gradients' definition takes the stored sum and the forward's mean and rstd, which are the unrounded sum's
    dy = st["dy"].double()
    xh = torch.einsum("ncg,n->ncg", s.to(st["x"].dtype).double() - mean.view(-1, 1, 1), rstd)
    w = torch.einsum("ncg,c->ncg", dy, st["gamma"].double())
    along = torch.einsum("ncg,ncg->n", w, xh) / n
    dv = w - (torch.einsum("ncg->n", w) / n).view(-1, 1, 1) - torch.einsum("ncg,n->ncg", xh, along)
    dx = torch.einsum("ncg,n->ncg", dv, rstd) + st["ds"].double()
    return y, s, dx, torch.einsum("ncg,ncg->c", dy, xh), torch.einsum("ncg->c", dy)


def _exact_rec(st):
    """Token after token, the sequences side by side; gradients by automatic differentiation."""
    train, C, G = st["op"] == "rec_train", st["C"], st["G"]
    edges = st["cu"].tolist()
    B, T, dev = len(edges) - 1, st["x"].shape[0], st["x"].device
    order = [list(range(edges[i], edges[i + 1]))[::-1 if st["reverse"] else 1] for i in range(B)]
    parts = st["packed"].double().requires_grad_(train)
    h0 = torch.zeros((B, C, G), device=dev, dtype=torch.float64) if st["h0"] is None else st["h0"].double()
    h0.requires_grad_(train)
    by_length = sorted(range(B), key=lambda i: -len(order[i]))  # the running ones come first
    h, states, rows, last = h0[torch.tensor(by_length, device=dev)], [], [], {}
    running = B
    steps = torch.tensor([[order[i][t] for i in by_length if t < len(order[i])] + [0] * sum(t >= len(order[i]) for i in by_length)
                          for t in range(len(order[by_length[0]]))], device=dev)
    for t in range(steps.shape[0]):
        alive = running
        while alive > 0 and len(order[by_length[alive - 1]]) <= t:
            alive -= 1
        if alive < running:
            for j in range(alive, running):
                last[by_length[j]] = h[j]
            h, running = h[:alive], alive
        at = steps[t, :alive]
        z = parts[at, C:2 * C]
        h = (torch.exp(z) * h + parts[at, :C]) / (1 + torch.exp(z))
        states.append(h)
        rows.append(at)
    for j in range(running):
        last[by_length[j]] = h[j]
    y = torch.empty((T, C, G), device=dev, dtype=torch.float64).index_copy(0, torch.cat(rows), torch.cat(states))
    if st["gate"]:
        o = parts[:, 2 * C:]
        y = y * o / (1 + torch.exp(-o))
    final = torch.stack([last[i] for i in range(B)])
    if not train:
        return y.detach(), final.detach()
    loss = (y * st["dy"].double()).sum()
    if st["dfinal"] is not None:
        loss = loss + (final * st["dfinal"].double()).sum()
    dparts, dh0 = torch.autograd.grad(loss, (parts, h0))
    outs = (y.detach(), final.detach(), dparts)
    return outs + (dh0,) if st["state"] else outs


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(st)
    if case["op"] == "rec_train" and case["len"] > 8192:
        return None
    return _exact_rec(st)
