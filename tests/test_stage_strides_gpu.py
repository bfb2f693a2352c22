"""GPU tests of strides that the stage operators take though they look odd: the same bits as with contiguous tensors."""
import pytest
import torch

import fourier_domain_linear_amd as eq
from test_attention_gpu import DT, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_whose_heads_lie_between_other_tokens(dtype, cuda_device):
    """Neither stride spans the other's whole extent, and yet no two heads share elements."""
    q, k, v, do, cu, _ = _inputs([3], [3], 2, 2, 64, dtype, cuda_device, seed=41)
    o, lse = eq.attention(q, k, v, cu, cu)
    grads = eq.attention_backward(do, q, k, v, o, lse, cu, cu)
    odd = lambda: torch.zeros((1024,), dtype=DT[dtype], device=cuda_device).as_strided((3, 2, 64), (128, 192, 1))  # noqa: E731
    out, dq, dk, dv = (odd() for _ in range(4))
    eq.attention(q, k, v, cu, cu, out=out)
    eq.attention_backward(do, q, k, v, out, lse, cu, cu, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    for a, b in zip((o, *grads), (out, dq, dk, dv)):
        assert torch.equal(a, b)
