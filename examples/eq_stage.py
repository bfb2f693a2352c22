"""One equivariant transformer stage on the library's operators: norm -> EQ-Linear (q, k, v) -> rotary positions ->
attention -> EQ-Linear -> norm with the residual -> MLP block -> norm with the residual, over packed images of different
sizes, forward and the gradients of its attention half.

    python examples/eq_stage.py            # p4, 192 channels, 12 heads, 16 images of 28 x 28: shapes and times

Tokens are x[N, C, G], group axis innermost; a head is dc channels x G. Turning an image a quarter (positions
(row, col) -> (-col, row)) and shifting the group axis by one shifts every output alike.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fourier_domain_linear_amd as eq  # noqa: E402


class Stage:
    """Weights of a stage: C channels, H heads of C / H channels, MLP width 4 C, group order G."""

    def __init__(self, C: int, H: int, G: int, dtype: torch.dtype, device, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *shape, std: (torch.randn(shape, generator=gen) * std).to(dtype).to(device)  # noqa: E731
        self.C, self.H, self.G, self.dc = C, H, G, C // H
        self.W = {"qkv": rand(3 * C, C, G, std=(C * G) ** -0.5), "out": rand(C, C, G, std=(C * G) ** -0.5),
                  "up": rand(4 * C, C, G, std=(C * G) ** -0.5), "down": rand(C, 4 * C, G, std=(4 * C * G) ** -0.5)}
        self.b = {n: rand(w.shape[0], std=0.1) for n, w in self.W.items()}
        self.gamma = [(1 + rand(C, std=0.1).float()).to(dtype) for _ in range(3)]
        self.layer = {n: eq.prepare_weights(w, backward=True) for n, w in self.W.items()}
        self.pairs = (self.dc // 4, self.dc // 2 - self.dc // 4)  # channel pairs of the rows and the columns

    def forward(self, x: torch.Tensor, pos: torch.Tensor, cu: torch.Tensor):
        """x [N, C, G] of images packed at the bounds cu, pos int32 [N, 2] -> (normalised output, residual stream,
        what the gradients need)."""
        N, H, dc, G = x.shape[0], self.H, self.dc, self.G
        y1, _, r1 = eq.rmsnorm(x, self.gamma[0])
        qkv = eq.forward(self.layer["qkv"], y1, self.b["qkv"]).view(N, 3 * H, dc, G)
        eq.rotary(qkv[:, :2 * H], pos, self.pairs, out=qkv[:, :2 * H])  # q and k, in place
        q, k, v = qkv.split(H, 1)
        o, lse = eq.attention(q, k, v, cu, cu)
        a = eq.forward(self.layer["out"], o.view(N, self.C, G), self.b["out"])
        y2, s2, r2 = eq.rmsnorm(a, self.gamma[1], residual=x)
        m = eq.mlp_block(self.layer["up"], self.b["up"], self.layer["down"], self.b["down"], y2)
        y3, s3, _ = eq.rmsnorm(m, self.gamma[2], residual=s2)
        return y3, s3, {"x": x, "y1": y1, "r1": r1, "qkv": qkv, "o": o, "lse": lse, "y2": y2, "s2": s2, "r2": r2}

    def attention_backward(self, dy2: torch.Tensor, ds2: torch.Tensor | None, pos: torch.Tensor, cu: torch.Tensor, kept: dict):
        """Gradients of the attention half from those of the second norm's outputs (y2, s2): (dx, weight gradients)."""
        N, H, dc, G = dy2.shape[0], self.H, self.dc, self.G
        da, dgamma2 = eq.rmsnorm_backward(dy2, kept["s2"], self.gamma[1], kept["r2"], ds=ds2)
        o = kept["o"].view(N, self.C, G)
        do = eq.backward_data(self.layer["out"], da).view(N, H, dc, G)
        dW_out, db_out = eq.backward_weights(self.layer["out"], o, da)
        q, k, v = kept["qkv"].split(H, 1)
        dqkv = torch.empty_like(kept["qkv"])
        dq, dk, dv = dqkv.split(H, 1)
        eq.attention_backward(do, q, k, v, kept["o"], kept["lse"], cu, cu, dq=dq, dk=dk, dv=dv)
        eq.rotary(dqkv[:, :2 * H], pos, self.pairs, inverse=True, out=dqkv[:, :2 * H])
        dqkv = dqkv.view(N, 3 * self.C, G)
        dy1 = eq.backward_data(self.layer["qkv"], dqkv)
        dW_qkv, db_qkv = eq.backward_weights(self.layer["qkv"], kept["y1"], dqkv)
        dx, dgamma1 = eq.rmsnorm_backward(dy1, kept["x"], self.gamma[0], kept["r1"], ds=da)
        return dx, {"qkv": dW_qkv, "out": dW_out, "b_qkv": db_qkv, "b_out": db_out, "gamma1": dgamma1, "gamma2": dgamma2}


def packed_images(sizes, device):
    """(pos int32 [N, 2], cu int32 [images + 1]) of images of sizes[i] = (height, width), one after the other."""
    pos = torch.cat([torch.cartesian_prod(torch.arange(h), torch.arange(w)).view(-1, 2) for h, w in sizes])
    cu = torch.tensor([0] + [h * w for h, w in sizes]).cumsum(0)
    return pos.to(torch.int32).to(device), cu.to(torch.int32).to(device)


def main():
    device = torch.device("cuda:0")
    stage = Stage(192, 12, 4, torch.bfloat16, device)
    pos, cu = packed_images([(28, 28)] * 16, device)
    x = torch.randn((pos.shape[0], 192, 4), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(device)
    dy, ds = torch.randn_like(x), torch.randn_like(x)

    def timed(call, n=20):
        call()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        begin.record()
        for _ in range(n):
            r = call()
        end.record()
        end.synchronize()
        return r, begin.elapsed_time(end) / n * 1e3

    (y, s, kept), forward_us = timed(lambda: stage.forward(x, pos, cu))
    (dx, grads), backward_us = timed(lambda: stage.attention_backward(dy, ds, pos, cu, kept))
    print(f"x {tuple(x.shape)} -> y {tuple(y.shape)}, residual {tuple(s.shape)}: {forward_us:.0f} us")
    print(f"dx {tuple(dx.shape)}, {', '.join(f'd{n} {tuple(g.shape)}' for n, g in grads.items())}: {backward_us:.0f} us")


if __name__ == "__main__":
    main()
