"""A whole transformer stage (examples/eq_stage.py) at the group orders 2 and 8: turning the images and shifting the group axis
commutes with it."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from eq_stage import Stage, packed_images  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bar", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)], ids=["f32", "bf16"])
@pytest.mark.parametrize("G,quarters", [(8, 1), (8, 3), (8, 2), (2, 2)])
def test_stage_commutes_with_turns(G, quarters, dtype, bar, cuda_device):
    """Bars: the layers' own parity bars (relative Frobenius 1e-5 and 1e-2) twice, for the two sides."""
    stage = Stage(32, 4, G, dtype, cuda_device)
    pos, cu = packed_images([(7, 9), (5, 4), (1, 1)], cuda_device)
    x = torch.randn((pos.shape[0], 32, G), generator=torch.Generator().manual_seed(3)).to(dtype).to(cuda_device)
    turned = pos
    for _ in range(quarters):
        turned = torch.stack([-turned[:, 1], turned[:, 0]], 1)
    shift = quarters * G // 4
    y, s, _ = stage.forward(x, pos, cu)
    y2, s2, _ = stage.forward(x.roll(shift, 2).contiguous(), turned.contiguous(), cu)
    for a, b in ((y, y2), (s, s2)):
        a, b = a.double().roll(shift, 2), b.double()
        assert float((a - b).norm() / a.norm()) <= bar
