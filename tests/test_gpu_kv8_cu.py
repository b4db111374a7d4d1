"""A cu that descends leaves a call over the 8-bit cache without work, in whatever
form the call has its items."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_fwd_kv8, attn_fwd_status
from test_gpu_kv8 import _dev, _random_cache, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("long_table", [False, True])
@pytest.mark.parametrize("B", [3, 40, 127, 129, 300, 5000])
def test_a_descending_cu_is_reported_and_costs_no_work(B, long_table):
    H, D, P, T = 2, 64, 16, 8
    cache, q = _random_cache(8, H, D, P, 4), _randn((T, 4, D), 8)
    lens, table = _dev([128] * B), _dev([list(range(8)) + [-1] * (5000 if long_table else 0)] * B)
    out, lse = torch.full((T, 4, D), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, 4), 5.0, device="cuda")
    spread = np.minimum(np.arange(B + 1), T)
    back = spread.copy()
    back[2] = 0  # (two requests share a token)
    late = np.r_[[0] * (B - 1), T, 3]  # the last request descends, the one before it has all tokens
    for cu in ([T * (i & 1) for i in range(B + 1)], back, late):
        attn_fwd_kv8(q, _dev(cu), lens, table, cache, P, out=out, lse=lse)
        assert attn_fwd_status() == -7
        assert (out == 5).all() and (lse == 5).all()
    attn_fwd_kv8(q, _dev([0] * (B - 1) + [T, T]), lens, table, cache, P, causal=False, out=out, lse=lse)
    assert attn_fwd_status() == 0 and (out != 5).any(-1).all() and (lse != 5).all() and torch.isfinite(lse).all()
