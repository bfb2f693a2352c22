"""Host-side checks of what workspace the attention asks for."""
import ctypes

import pytest

import fourier_domain_linear_amd as eq
from test_stage_abi import _args


@pytest.mark.parametrize("tokens, group", [(1, 8), (4, 8), (8, 4), (32, 1)])
def test_few_rows_over_a_cache_need_parts_of_chunks_alone(tokens, group):
    """Up to 32 packed rows in all are the chunks' kernel's; nothing is set aside for row tiles that none of them takes. A chunk
    has at least 128 keys, and its part of a row the head's values with a maximum and a sum."""
    lib, keys, heads, dim = eq.load_library(), 20000, 2, 128
    a = _args(total_q=tokens, total_k=keys, heads_q=group * heads, heads_kv=heads, dim=dim)
    need = lib.eqlin_attention_workspace(ctypes.byref(a))
    rows = group if tokens == 1 else 32
    assert 0 < need <= (keys // 128 + 1) * heads * rows * (dim + 2) * 4
