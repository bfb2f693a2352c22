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


def _one(t, dim, stride):
    """t with another stride of a dimension of size one, which no element's place depends on."""
    assert t.shape[dim] == 1
    strides = list(t.stride())
    strides[dim] = stride
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("stride", [1, 1 << 30], ids=["odd", "far"])
def test_strides_of_single_tokens_and_heads_mean_nothing(stride, cuda_device):
    """A tensor of one token or one head may have any stride there (a transposed cache of one head, a slice of a long one)."""
    dev = cuda_device
    for lq, lk, Hq, Hkv in ((1, 1, 4, 2), (5, 700, 1, 1), (1, 700, 3, 1)):
        q, k, v, do, cu_q, cu_k = _inputs([lq], [lk], Hq, Hkv, 64, "bf16", dev, seed=42)
        o, lse = eq.attention(q, k, v, cu_q, cu_k)
        grads = eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k)

        def odd(t):
            for dim in (0, 1):
                t = _one(t, dim, stride) if t.shape[dim] == 1 else t
            return t

        out = odd(torch.zeros_like(o))
        dq, dk, dv = (odd(torch.zeros_like(t)) for t in (q, k, v))
        eq.attention(odd(q), odd(k), odd(v), cu_q, cu_k, out=out)
        eq.attention_backward(odd(do), odd(q), odd(k), odd(v), out, lse, cu_q, cu_k, dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        for a, b in zip((o, *grads), (out, dq, dk, dv)):
            assert torch.equal(a, b)
    for N, H in ((1, 3), (6, 1), (1, 1)):
        x = torch.randn((N, H, 16, 4), generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).to(dev)
        pos = torch.arange(2 * N, dtype=torch.int32, device=dev).view(N, 2)
        y = eq.rotary(x, pos, (4, 4))
        z = x
        for dim in (0, 1):
            z = _one(z, dim, stride) if z.shape[dim] == 1 else z
        assert torch.equal(eq.rotary(z, pos, (4, 4)), y)
        eq.rotary(z, pos, (4, 4), out=x)  # in place, by another view
        assert torch.equal(x, y)
