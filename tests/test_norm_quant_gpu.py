"""GPU test of the 8-bit norm's codes at ties: q is y / scale, divided, to the nearest even."""
import numpy as np
import pytest
import torch

import fourier_domain_linear_amd as eq
from oracle import stage

pytestmark = pytest.mark.gpu


# (C, G): rows in registers of one wave and of four, and the element form
@pytest.mark.parametrize("C,G", [(64, 4), (512, 8), (131, 1)])
def test_codes_at_ties(C, G, cuda_device):
    """Rows whose values over the scale lie on the points halfway between two codes up to fp32 rounding, so that the last bit of the
    quotient decides: the codes are those of fp32's y = s rstd, the scale max |y| / 448 and the quotient y / scale, each rounded
    once, from the kernel's own rstd. Bar: none, every code and scale is equal."""
    rows, gen = 256, np.random.default_rng(C)
    code = stage._E4M3[1:]
    ties = (code[:-1] + code[1:]) / 2  # exact in fp32
    x = gen.choice(ties, (rows, C, G)) * gen.choice([-1.0, 1.0], (rows, C, G))
    x[:, 0, 0] = 448
    x = (x * gen.uniform(0.5, 2.0, (rows, 1, 1))).astype(np.float32)
    q, scale, s, rstd = eq.rmsnorm_quant(torch.from_numpy(x).to(cuda_device), eps=0.0)
    torch.cuda.synchronize()
    y = x * rstd.cpu().numpy()[:, None, None]
    want_scale = np.abs(y).max(axis=(1, 2)) / np.float32(448)
    assert y.dtype == want_scale.dtype == np.float32
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    want = stage.e4m3_nearest(y / want_scale[:, None, None])
    got = q.float().cpu().numpy()
    print(f"[parity] C={C} G={G}: {(got != want).sum()} of {got.size} codes differ", flush=True)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("C,G", [(64, 4), (512, 8), (131, 1)])
def test_an_infinite_scale(C, G, cuda_device):
    """A row with an infinite value has an infinite scale; its finite values are 0 and the infinite ones NaN."""
    x = torch.randn((3, C, G), generator=torch.Generator().manual_seed(C)).to(cuda_device)
    gamma = torch.ones(C, device=cuda_device)
    gamma[2] = float("inf")
    q, scale, _, _ = eq.rmsnorm_quant(x, gamma)
    torch.cuda.synchronize()
    codes = q.float()
    assert bool(scale.isinf().all()) and bool(codes[:, 2].isnan().all())
    codes[:, 2] = 0
    assert not codes.any()
