"""One equivariant recurrent stage on the library's operators: layer norm -> EQ-Linear (values, forget gates, output gates) -> gated
recurrence over each sequence's tokens -> EQ-Linear -> layer norm with the residual -> MLP block -> layer norm with the
residual. Whole packed sequences, forward and the gradients of the mixing half, or one new token in each of many streams, whose
states are kept from call to call.

    python examples/eq_recurrent_stage.py      # p4, 192 channels, 16 sequences of 784 tokens, then 64 streams: shapes and times

Tokens are x[N, C, G], group axis innermost; every operator commutes with a shift of it. (The recurrence goes along the tokens as they
are packed, so turning an image commutes with the stage only as far as its tokens' order does.)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fourier_domain_linear_amd as eq  # noqa: E402


class RecurrentStage:
    """Weights of a stage: C channels, MLP width 4 C, group order G; reverse: the recurrence runs from the last token on."""

    def __init__(self, C: int, G: int, dtype: torch.dtype, device, reverse: bool = False, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *shape, std: (torch.randn(shape, generator=gen) * std).to(dtype).to(device)  # noqa: E731
        self.C, self.G, self.reverse = C, G, reverse
        self.W = {"mix": rand(3 * C, C, G, std=(C * G) ** -0.5), "out": rand(C, C, G, std=(C * G) ** -0.5),
                  "up": rand(4 * C, C, G, std=(C * G) ** -0.5), "down": rand(C, 4 * C, G, std=(4 * C * G) ** -0.5)}
        self.b = {n: rand(w.shape[0], std=0.1) for n, w in self.W.items()}
        # channels remember for one token to some hundreds
        self.b["mix"][C:2 * C] += torch.linspace(0, 6, C).to(dtype).to(device)
        self.gamma = [(1 + rand(C, std=0.1).float()).to(dtype) for _ in range(3)]
        self.beta = [rand(C, std=0.1) for _ in range(3)]
        self.layer = {n: eq.prepare_weights(w, backward=True) for n, w in self.W.items()}

    def forward(self, x: torch.Tensor, cu: torch.Tensor, state: torch.Tensor | None = None, longest: int | None = None,
                training: bool = False):
        """x [N, C, G] of sequences packed at the bounds cu (from 0 to N: rows of no sequence would come out of the recurrence
        unwritten), state float32 [batch, C, G] -> (normalised output, residual stream, states after the last tokens, what the
        gradients need)."""
        C = self.C
        y1, _, m1, r1 = eq.layernorm(x, self.gamma[0], self.beta[0])
        mix = eq.forward(self.layer["mix"], y1, self.b["mix"])
        v, f, o = mix[:, :C], mix[:, C:2 * C], mix[:, 2 * C:]
        h, final, marks = eq.recurrence(v, f, cu, gate=o, state=state, reverse=self.reverse, longest=longest, with_marks=training)
        a = eq.forward(self.layer["out"], h, self.b["out"])
        y2, s2, m2, r2 = eq.layernorm(a, self.gamma[1], self.beta[1], residual=x)
        m = eq.mlp_block(self.layer["up"], self.b["up"], self.layer["down"], self.b["down"], y2)
        y3, s3, _, _ = eq.layernorm(m, self.gamma[2], self.beta[2], residual=s2)
        return y3, s3, final, {"x": x, "y1": y1, "m1": m1, "r1": r1, "mix": mix, "h": h, "marks": marks, "y2": y2, "s2": s2, "m2": m2, "r2": r2}

    def mix_backward(self, dy2: torch.Tensor, ds2: torch.Tensor | None, cu: torch.Tensor, kept: dict, dfinal: torch.Tensor | None = None,
                     longest: int | None = None):
        """Gradients of the mixing half from those of the second norm's outputs (y2, s2) and of the final states: (dx, dstate,
        weight gradients)."""
        C = self.C
        da, dgamma2, dbeta2 = eq.layernorm_backward(dy2, kept["s2"], self.gamma[1], kept["m2"], kept["r2"], ds=ds2)
        dh = eq.backward_data(self.layer["out"], da)
        dW_out, db_out = eq.backward_weights(self.layer["out"], kept["h"], da)
        mix = kept["mix"]
        dmix = torch.empty_like(mix)
        _, _, _, dstate = eq.recurrence_backward(dh, mix[:, :C], mix[:, C:2 * C], cu, kept["marks"], gate=mix[:, 2 * C:],
                                                 reverse=self.reverse, dfinal=dfinal, longest=longest, with_state=True, dx=dmix[:, :C],
                                                 dforget=dmix[:, C:2 * C], dgate=dmix[:, 2 * C:])
        dy1 = eq.backward_data(self.layer["mix"], dmix)
        dW_mix, db_mix = eq.backward_weights(self.layer["mix"], kept["y1"], dmix)
        dx, dgamma1, dbeta1 = eq.layernorm_backward(dy1, kept["x"], self.gamma[0], kept["m1"], kept["r1"], ds=da)
        return dx, dstate, {"mix": dW_mix, "out": dW_out, "b_mix": db_mix, "b_out": db_out, "gamma1": dgamma1, "beta1": dbeta1,
                            "gamma2": dgamma2, "beta2": dbeta2}


def main():
    device = torch.device("cuda:0")
    stage = RecurrentStage(192, 4, torch.bfloat16, device)
    cu = torch.arange(0, 16 * 784 + 1, 784, device=device, dtype=torch.int32)
    x = torch.randn((16 * 784, 192, 4), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(device)
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

    (y, s, final, kept), us = timed(lambda: stage.forward(x, cu, longest=784, training=True))
    print(f"x {tuple(x.shape)} -> y {tuple(y.shape)}, states {tuple(final.shape)}: {us:.0f} us")
    (dx, _, grads), us = timed(lambda: stage.mix_backward(dy, ds, cu, kept, longest=784))
    print(f"dx {tuple(dx.shape)}, {', '.join(f'd{n} {tuple(g.shape)}' for n, g in grads.items())}: {us:.0f} us")
    token, one = x[:64].contiguous(), torch.arange(65, device=device, dtype=torch.int32)
    state = torch.zeros((64, 192, 4), device=device)
    (y, _, _, _), us = timed(lambda: stage.forward(token, one, state=state, longest=1))
    print(f"one token in each of 64 streams -> y {tuple(y.shape)}: {us:.0f} us")


if __name__ == "__main__":
    main()
