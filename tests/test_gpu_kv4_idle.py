"""Attention over the 4-bit cache for batches of fixed slots of which few are
active: results, and that idle slots between the active ones cost no walk."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_fwd_kv4, attn_fwd_status, attn_kv4_append, attn_kv4_cache

pytestmark = pytest.mark.gpu

D, P, H, Hq = 64, 16, 2, 8


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _cache(pages, seed):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((pages * P, H, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    cache = attn_kv4_cache(pages, H, D, P)
    attn_kv4_append(k, v, _dev(range(pages * P)), cache, P)
    return cache


def _batch(B, active, lens, nq, width, pages, seed):
    """A batch of B slots, its idle ones with lengths and tables of their own; and the active requests alone."""
    r = np.random.default_rng(seed)
    all_nq, all_lens = np.zeros(B, dtype=np.int64), r.integers(0, width * P + 1, B)
    all_nq[active], all_lens[active] = nq, lens
    table = r.integers(0, pages, (B, width))
    q = torch.randn((int(sum(nq)), Hq, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    cu, few = np.concatenate([[0], np.cumsum(all_nq)]), np.concatenate([[0], np.cumsum(nq)])
    return ((q, _dev(cu), _dev(all_lens), _dev(table)),
            (q, _dev(few), _dev(lens), _dev(table[active].reshape(len(active), width))))


@pytest.mark.parametrize("width", [20, 3000])  # one cluster an item, and cut pieces
@pytest.mark.parametrize("B,active", [(33, [0, 32]), (129, [128]), (400, [0, 1, 200, 399]), (400, [399]),
                                      (2000, [3, 1000, 1001, 1999]),
                                      (16384, [0, 16383]),
                                      (16384, [8000, 8001, 16000])], ids=str)
def test_few_active_slots(B, active, width):
    cache = _cache(64, 1)
    r = np.random.default_rng(B)
    lens, nq = r.integers(1, 20 * P, len(active)), r.integers(1, 4, len(active))
    batch, alone = _batch(B, active, lens, nq, width, 64, 2)
    o, lse = attn_fwd_kv4(*batch, cache, P)
    want, wl = attn_fwd_kv4(*alone, cache, P)
    assert attn_fwd_status() == 0
    # the same keys, perhaps in other parts: a weight's half precision and the outputs' own rounding
    assert ((o.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -8).all()
    assert (lse - wl).abs().max() <= 2.0 ** -16


def test_bad_idle_slots_are_reported():
    # a length past the table in a slot without query tokens, before and after the active one
    cache = _cache(8, 3)
    for B in (40, 3000):
        for bad in (0, B - 1):
            batch, _ = _batch(B, [B // 2], [30], [1], 4, 8, 4)
            batch[2][bad] = 4 * P + 1
            attn_fwd_kv4(*batch, cache, P)
            assert attn_fwd_status() == -7
            batch[2][bad] = 4 * P
            attn_fwd_kv4(*batch, cache, P)
            assert attn_fwd_status() == 0


def _time(call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(10):
            call()
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best / 10


@pytest.mark.parametrize("tokens", [300, 330])  # (330: the second item begins inside a warp's piece)
@pytest.mark.parametrize("width", [25, 3000])
def test_idle_slots_cost_no_walk(width, tokens):
    # two active slots at the ends of the largest batch: the lengths are read by all threads of a CTA, not by one warp
    # (some 200 us) or, between an item and the next, by one load after the other (2.5 ms)
    g = torch.Generator().manual_seed(5)
    k = torch.randn((64 * P, 1, D), generator=g).to(torch.bfloat16).cuda()
    cache = attn_kv4_cache(64, 1, D, P)
    attn_kv4_append(k, k, _dev(range(64 * P)), cache, P)
    batch, _ = _batch(16384, [0, 16383], [tokens, tokens], [1, 1], width, 64, 6)
    out, lse = attn_fwd_kv4(*batch, cache, P)
    assert _time(lambda: attn_fwd_kv4(*batch, cache, P, out=out, lse=lse)) <= (0.12 if width == 25 else 0.5)  # ms
