"""Attention over the 8-bit cache with scores far from zero.

Where all tokens that count have the same score, or one is far above the others, the
weights do not depend on how large the scores are, and neither may the error of O:

  weights exp2 2^-22 relative, its argument's roundings (numbers below 512: 2^-16
          relative), four parts of 4 bits 2^-16 relative or 2^-29 of the row's largest
          weight times V's scale, times codes up to 448
  output  float32 sums, cut at 2^-23 once for each 32 tokens, merged (2^-20), one
          rounding to bfloat16: 2^-8 (half a step is 2^-9)
so |dO| <= (2^-14 + n 2^-28) A + 2^-29 448 n B + 2^-8 |O|, A = mean |V| of the n tokens that
count, B = the largest scale of V over n.  A token that counts alone is V itself: V is a
bfloat16 number, and 2^-14 is below half of a bfloat16 step.

LSE is a float32 number: the score's factors, the sum and the change of base are half a
dozen roundings of 2^-24, so |dLSE| <= 2^-21 |LSE| + 2^-20."""
import math

import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_fwd_kv8, attn_fwd_status, attn_kv8_append, attn_kv8_cache, attn_kv8_read
from exact_attention_attn_gb300.workloads import to_f64

pytestmark = pytest.mark.gpu

# head dim, query heads of a kv head: every number of rows of a tile
SHAPES = [(64, 4), (128, 3), (192, 4), (256, 4), (64, 7), (128, 8), (192, 8), (256, 5), (64, 16), (128, 12), (192, 16), (256, 28), (64, 28), (128, 32)]
P = 16


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _cache(k, v):
    """A cache of the tokens, and what it holds for them: V as float64 [n, H, D] and the scale of V of each token [n, H]."""
    n, H, D = k.shape
    cache = attn_kv8_cache(-(-n // P), H, D, P)
    slots = _dev(np.arange(n))
    attn_kv8_append(k, v, slots, cache, P)
    _, held = attn_kv8_read(slots, cache, P)
    tail = cache[..., P * D:].reshape(-1, H, 16 * D + 16)[..., 16 * D + 4:16 * D + 8].contiguous().view(torch.float32)
    return cache, to_f64(held).transpose(1, 0, 2), np.repeat(to_f64(tail)[..., 0], 16, 0)[:n]


def _attend(q, cache, lens, long_table, scale, causal=True):
    """One query token a request, each request the first lens[r] tokens of the cache."""
    B = len(lens)
    pages = cache.shape[0]
    table = np.full((B, 80000 // P if long_table else pages), -1)
    table[:, :pages] = np.arange(pages)
    o, l = attn_fwd_kv8(q, _dev(np.arange(B + 1)), _dev(lens), _dev(table), cache, P, scale=scale, causal=causal)
    assert attn_fwd_status() == 0
    return to_f64(o), to_f64(l)


def _check_mean(o, v, unit):
    """o [heads, D]: the mean of v [n, D]."""
    n = len(v)
    O, A = v.mean(0), np.abs(v).mean(0)
    tol = (2.0 ** -14 + n * 2.0 ** -28) * A + 2.0 ** -29 * 448 * unit.max() + 2.0 ** -8 * np.abs(O)
    err = np.abs(o - O)
    assert (err <= tol).all(), (err / tol).max()


def _values(n, D, seed, exps):
    """bfloat16 [n, 1, D], blocks of 16 tokens of sizes 2^exps in turn."""
    x = torch.randn((n, 1, D), generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    size = 2.0 ** torch.tensor([float(exps[i // 16 % len(exps)]) for i in range(n)], dtype=torch.float64)
    return (x.clamp(-3, 3) * size[:, None, None]).to(torch.bfloat16).cuda()


def _one_dim(n, D, value):
    x = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    x[..., D - 5] = value
    return x


def _scores(power, sign):
    """q and K whose product is about sign 2^power, both bfloat16 numbers (K an e4m3 number times a power of two)."""
    a = power // 2
    return 1.3125 * 2.0 ** a * sign, 1.25 * 2.0 ** (power - a), 1.3125 * 1.25 * 2.0 ** power * sign


POWERS = [10, 20, 24, 25, 27, 30, 41, 60, 100, 124]


@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("long_table", [False, True])
def test_one_token_is_its_value(D, group, long_table):
    for exp in (-90, -7, 0, 1, 30, 117):
        v = _values(1, D, D + exp, [exp])
        for power in POWERS:
            for sign in (1, -1):
                a, b, s = _scores(power, sign)
                cache, held, _ = _cache(_one_dim(1, D, b), v)
                q = _one_dim(1, D, a).expand(1, group, D).contiguous()
                o, l = _attend(q, cache, [1], long_table, 1.0)
                assert (np.abs(l - s) <= 2.0 ** -21 * abs(s) + 2.0 ** -20).all(), (exp, power, sign, l[0, 0], s)
                assert np.array_equal(o[0], np.broadcast_to(held[0], o[0].shape)), (exp, power, sign)


@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("long_table", [False, True])
@pytest.mark.parametrize("exps", [[-7, -8], [0, -6, 3, -100], [5, 100, 40]])
def test_equal_tokens_have_equal_weights(D, group, long_table, exps):
    # of one block, of blocks of one tile with other scales, of several tiles, of cut items and of clusters
    lens = [2, 17, 40, 200, 700, 1500]
    n = max(lens)
    v = _values(n, D, D, exps)
    for power in POWERS:
        for sign in (1, -1):
            a, b, s = _scores(power, sign)
            cache, held, unit = _cache(_one_dim(n, D, b), v)
            q = _one_dim(len(lens), D, a).expand(len(lens), group, D).contiguous()
            o, l = _attend(q, cache, lens, long_table, 1.0)
            for r, m in enumerate(lens):
                L = s + math.log(m)
                assert (np.abs(l[r] - L) <= 2.0 ** -21 * abs(L) + 2.0 ** -20).all(), (power, sign, m)
                _check_mean(o[r], held[:m, 0], unit[:m, 0])


@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("long_table", [False, True])
def test_a_heavy_token_among_others(D, group, long_table):
    # its score is far above the others', whose V are far larger or far smaller
    n = 600
    for where in (0, 130, 599):
        for exps in ([-30, 40], [50, -5]):
            v = _values(n, D, where, exps)
            for power in POWERS[1:]:
                for sign in (1, -1):
                    a, b, s = _scores(power, sign)
                    k = _one_dim(n, D, b if sign < 0 else -b)  # the others' scores are -|s|
                    k[where] *= -1
                    cache, held, _ = _cache(k, v)
                    q = _one_dim(1, D, a).expand(1, group, D).contiguous()
                    o, l = _attend(q, cache, [n], long_table, 1.0)
                    assert (np.abs(l - abs(s)) <= 2.0 ** -21 * abs(s)).all(), (where, power, sign)
                    assert np.array_equal(o[0], np.broadcast_to(held[where], o[0].shape)), (where, power, sign, exps)


@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("long_table", [False, True])
def test_large_q_and_large_k_whose_scores_are_small(D, group, long_table):
    # their largest values' product passes 2^128: in dims where the other one is zero, cancelling, or of other tokens of the block
    n, half = 200, D // 2
    v = _values(n, D, 1, [0, 2])
    q = torch.zeros((3, group, D), dtype=torch.bfloat16, device="cuda")
    q[0, :, :half] = 2.0 ** 80
    q[1, :, 3], q[1, :, 9] = 2.0 ** 90, 2.0 ** 90
    q[2, :, 0] = -1.5 * 2.0 ** 99
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[:, :, half:] = 1.75 * 2.0 ** 80
    k[::3, :, half:] *= -1
    k[:, :, 3], k[:, :, 9] = 2.0 ** 70, -(2.0 ** 70)
    for rows in (slice(0, n), slice(5, n, 16)):  # (or all but one token in each block are zero)
        x = torch.zeros_like(k)
        x[rows] = k[rows]
        cache, held, unit = _cache(x, v)
        o, l = _attend(q, cache, [n, n, n], long_table, 0.5)
        for r in range(3):
            assert (np.abs(l[r] - math.log(n)) <= 2.0 ** -20 * (1 + math.log(n))).all(), (r, l[r])
            _check_mean(o[r], held[:, 0], unit[:, 0])


@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("long_table", [False, True])
def test_scores_next_to_the_end_of_float32(D, group, long_table):
    # up to 2^127, next to -2^127 too, where "no token yet" must not be taken for a reference
    lens = [1, 16, 129, 700]
    n = max(lens)
    v = _values(n, D, 1, [-7, -5])
    for a, b in ((2.0 ** 63, 2.0 ** 60), (2.0 ** 63, 1.25 * 2.0 ** 61), (2.0 ** 63, 1.5 * 2.0 ** 63), (2.0 ** 63, 1.875 * 2.0 ** 63)):
        for sign in (1, -1):
            s = sign * a * b
            cache, held, unit = _cache(_one_dim(n, D, b), v)
            q = _one_dim(len(lens), D, a * sign).expand(len(lens), group, D).contiguous()
            o, l = _attend(q, cache, lens, long_table, 1.0)
            for r, m in enumerate(lens):
                assert (np.abs(l[r] - s) <= 2.0 ** -21 * abs(s)).all(), (s, m, l[r])
                _check_mean(o[r], held[:m, 0], unit[:m, 0])


@pytest.mark.parametrize("D,group", SHAPES)
def test_rows_that_see_no_token_beside_scores_far_below_zero(D, group):
    # three query tokens of two cached ones: the first sees none, the others' scores are -2^126
    v = _values(2, D, 3, [0])
    cache, held, _ = _cache(_one_dim(2, D, 2.0 ** 63), v)
    table = _dev([[0]])
    q = _one_dim(3, D, -(2.0 ** 63)).expand(3, group, D).contiguous()
    o, l = attn_fwd_kv8(q, _dev([0, 3]), _dev([2]), table, cache, P, scale=1.0)
    assert attn_fwd_status() == 0
    o, l = to_f64(o), to_f64(l)
    assert (o[0] == 0).all() and np.isneginf(l[0]).all()
    assert np.array_equal(o[1], np.broadcast_to(held[0], o[1].shape)) and (np.abs(l[1:] + 2.0 ** 126) <= 2.0 ** 105).all()
    _check_mean(o[2], held[:, 0], np.array([0.0]))
