"""GPU test that a row's result has no part, to the bit, of keys that it does not see and of rows beside it."""
import pytest
import torch

import fourier_domain_linear_amd as eq
from test_attention_gpu import _inputs

pytestmark = pytest.mark.gpu


# (query lengths, key lengths, Hq, Hkv, D): prompts, a prompt over many keys (split), steps
CASES = {"prompt": ([300, 20], [300, 20], 4, 2, 64), "wide": ([200], [260], 2, 2, 128), "split": ([40], [3000], 7, 7, 128),
         "step": ([4, 3], [700, 1300], 8, 2, 64), "narrow": ([90], [90], 3, 1, 24)}


@pytest.mark.parametrize("late", [30.0, 1000.0, float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_later_keys_have_no_part(name, dtype, late, cuda_device):
    """The last two tokens of each causal sequence get keys far larger than the others, or infinite: scores that raise the running
    maximum of the rows that see them. Every other row keeps its bits, in o, lse and dq."""
    lq, lk, Hq, Hkv, D = CASES[name]
    q, k, v, do, cu_q, cu_k = _inputs(lq, lk, Hq, Hkv, D, dtype, cuda_device, seed=51)

    def run(k):
        o, lse = eq.attention(q, k, v, cu_q, cu_k, causal=True)
        return o, lse, eq.attention_backward(do, q, k, v, o, lse, cu_q, cu_k, causal=True)[0]

    k2, keep = k.clone(), torch.ones(sum(lq), dtype=torch.bool)
    for i in range(len(lq)):
        k2[sum(lk[:i + 1]) - 2:sum(lk[:i + 1])] *= late
        keep[sum(lq[:i + 1]) - 2:sum(lq[:i + 1])] = False
    for a, b in zip(run(k), run(k2)):
        torch.cuda.synchronize()
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_beside_have_no_part(dtype, cuda_device):
    """Rows of one sequence whose queries grow a hundredfold leave the others' bits alone."""
    q, k, v, do, cu_q, cu_k = _inputs([64], [200], 2, 1, 64, dtype, cuda_device, seed=52)
    q2 = q.clone()
    q2[1::2] *= 100
    for a, b in zip(eq.attention(q, k, v, cu_q, cu_k), eq.attention(q2, k, v, cu_q, cu_k)):
        torch.cuda.synchronize()
        assert torch.equal(a[::2], b[::2])
