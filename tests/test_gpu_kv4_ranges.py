"""Attention over the 4-bit cache where V's sizes differ by many powers of two:
tokens that a row does not see, or gives no weight, must not take the bits of
those that count.

Tolerance, per element: that of test_gpu_kv4 (scores dS = 2^-18 max_j Sabs; weights
2^-11 of A = sum_j p_j (s_j c_j + |m_j|), exp2 and float32 sums 2^-19 A, one rounding
to bfloat16 2^-8 |O|), and for products p_j s_j too small for half precision's normal
range an absolute error each, times a code up to 15, of 2^-28 of the row's sum of
them: a row's products are scaled so that the largest, or a sixteenth of the sum of
p s c, reaches 2^3, and half a step of the subnormals is 2^-25."""
import math

import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_fwd_kv4, attn_fwd_status, attn_kv4_append, attn_kv4_cache
from exact_attention_attn_gb300.workloads import to_f64
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _check(out, lse, q, n, cache, D, P, causal=True):
    """One request whose tokens are the cache's first n, in order."""
    nq, Hq = q.shape[:2]
    H, G, scale = cache.shape[1], D // 64, D ** -0.5
    (kc, ks, km), (vc, vs, vm) = ([x.transpose(1, 0, 2, 3).reshape(H, -1, x.shape[3])[:, :n] for x in side]
                                  for side in S.kv4_unpack(cache.cpu().numpy(), D, P))
    k, v = S.kv4_values(kc, ks, km), S.kv4_values(vc, vs, vm)
    ka, va = S.kv4_values(kc, ks, np.abs(km)), S.kv4_values(vc, vs, np.abs(vm))
    qf, got, gl = to_f64(q), to_f64(out), to_f64(lse)
    for t in range(nq):
        seen = min(n, max(0, t + 1 + n - nq)) if causal else n
        for hq in range(Hq):
            h = hq // (Hq // H)
            x = scale * (k[h, :seen] @ qf[t, hq])
            top = x.max()
            p = np.exp(x - top)
            L = top + math.log(p.sum())
            p /= p.sum()
            want, A = p @ v[h, :seen], p @ va[h, :seen]
            dS = 2.0 ** -18 * scale * (ka[h, :seen] @ np.abs(qf[t, hq])).max()
            small = np.repeat(15 * seen * 2.0 ** -28 * (p @ vs[h, :seen]), 64)
            tol = (2.0 ** -11 + 2 * dS + 2.0 ** -19) * A + small + 2.0 ** -8 * np.abs(want)
            err = np.abs(got[t, hq] - want)
            assert (err <= tol).all(), (t, hq, (err / tol).max(), err.max(), np.abs(want).max())
            assert abs(gl[t, hq] - L) <= dS + 2.0 ** -20 * (1 + abs(L)), (t, hq, gl[t, hq], L)
    assert G == vs.shape[2]


def _run(k, v, q, P, wide=False, causal=True):
    """k, v [n, H, D] and q [nq, Hq, D], float32: one request (a wide table makes the call cut its items)."""
    n, H, D = k.shape
    pages = -(-n // P)
    cache = attn_kv4_cache(pages, H, D, P)
    k, v, q = (x.to(torch.bfloat16).cuda() for x in (k, v, q))
    attn_kv4_append(k, v, _dev(range(n)), cache, P)
    table = _dev([list(range(pages)) + [-1] * (80000 // P if wide else 0)])
    out, lse = attn_fwd_kv4(q, _dev([0, q.shape[0]]), _dev([n]), table, cache, P, causal=causal)
    torch.cuda.synchronize()
    assert attn_fwd_status() == 0
    _check(out, lse, q, n, cache, D, P, causal)
    return out


def _randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _scored(scores, H, D, seed):
    """K whose product with a query of ones, over sqrt(D), is about `scores` [n]."""
    k = torch.as_tensor(scores, dtype=torch.float32)[:, None, None] / math.sqrt(D)
    return k.expand(-1, H, D) + 0.05 * _randn((len(scores), H, D), seed)


SHAPES = [
    # D, P, Hq, Hkv
    (64, 16, 4, 1), (128, 16, 8, 2), (128, 64, 4, 1), (192, 32, 3, 1), (256, 16, 8, 2), (256, 64, 2, 1)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("power", [12, 40, 90])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_hidden_token_takes_no_bits(shape, power, wide):
    # V of the last tokens is 2^power times the others': the earlier query tokens must not notice
    D, P, Hq, H = shape
    n, nq = 75, 4
    k, v, q = _randn((n, H, D), 1), _randn((n, H, D), 2), _randn((nq, Hq, D), 3)
    out = _run(k, v, q, P, wide)
    big = v.clone()
    big[-1] *= 2.0 ** power
    big[-2, 0, :64] *= 2.0 ** (power + 7)
    got = _run(k, big, q, P, wide)
    # what the first two query tokens see is the same, so their outputs differ by roundings of half precision at most
    assert ((got[:2].float() - out[:2].float()).abs() <= 2.0 ** -7 * out[:2].float().abs() + 2.0 ** -9).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("P,D", [(16, 64), (64, 64), (16, 128), (32, 128)])
def test_hidden_tokens_of_a_tile_of_many_rows(P, D, wide):
    # more than 64 query rows a request: tiles of 16 rows, whose last tokens grow by 2^4 each
    n, nq = 90, 20
    k, v, q = _randn((n, 1, D), 4), _randn((n, 1, D), 5), _randn((nq, 4, D), 6)
    v[-nq:] *= 2.0 ** (4 * torch.arange(nq))[:, None, None]
    _run(k, v, q, P, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("at", [0, 17, 200, 299])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_token_of_no_weight_takes_no_bits(shape, at, wide):
    # a visible token 2^60 times as large whose weight is about e^-120, so that it adds nothing
    D, P, Hq, H = shape
    n = 300
    scores = _randn((n,), 7)
    scores[at] = -120.0
    k, v, q = _scored(scores, H, D, 8), _randn((n, H, D), 9), torch.ones((1, Hq, D))
    v[at] *= 2.0 ** 60
    _run(k, v, q, P, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("at", [0, 40, 149])
@pytest.mark.parametrize("D,P", [(64, 32), (128, 16), (256, 32)])
def test_a_small_weight_of_a_large_value_counts(D, P, at, wide):
    # weight 2^-50, values 2^52: this token's part of the output is a few times the others'
    n = 150
    scores = 0.3 * _randn((n,), 10)
    scores[at] = -50 * math.log(2.0) + math.log(n)
    k, v, q = _scored(scores, 1, D, 11), _randn((n, 1, D), 12), torch.ones((1, 4, D))
    v[at] *= 2.0 ** 52
    _run(k, v, q, P, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (192, 16)])
def test_rows_of_a_tile_that_weigh_a_large_value_differently(D, P, wide):
    # some heads look at the large tokens alone, others not at all, for one of V's groups
    n, big = 140, [3, 70, 139]
    scores = torch.zeros(n)
    scores[big] = 40.0
    k, v = _scored(scores, 1, D, 13), _randn((n, 1, D), 14)
    v[big, :, -64:] *= 2.0 ** 45
    q = torch.tensor([1.0, -1.0, 0.5, -0.25, 0.0, 2.0])[None, :, None].expand(1, 6, D)
    _run(k, v, q, P, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("up", [1, -1])
@pytest.mark.parametrize("D,P", [(64, 64), (128, 16), (256, 16)])
def test_values_that_fall_while_scores_rise(D, P, up, wide):
    # over 600 tokens the scores climb by 90 and V falls by 2^80 (or the other way round): every unit moves a reference
    n = 600
    ramp = torch.linspace(0, 1, n)
    k = _scored(90 * (ramp if up > 0 else 1 - ramp), 1, D, 15)
    v = _randn((n, 1, D), 16) * torch.exp2(80 * (1 - ramp if up > 0 else ramp))[:, None, None]
    _run(k, v, torch.ones((1, 4, D)), P, wide)
    _run(k, v, torch.ones((3, 4, D)), P, wide)


@pytest.mark.parametrize("wide", [False, True])
def test_groups_without_a_scale_beside_large_ones(wide):
    # constant V (scale 0) in most tokens, in one group in all of them
    n, D, P = 200, 128, 16
    k, v = _randn((n, 2, D), 17), _randn((n, 2, D), 18)
    v[:, :, 64:] = 1.5
    v[:150, 0] = -0.75
    v[60, 1, :64] *= 2.0 ** 70
    _run(k, v, _randn((4, 8, D), 19), P, wide)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_values_near_the_largest_number(shape, wide):
    # |V| up to 2^126: sums of weighted values must not pass float32 before they are divided by the weights' sum
    D, P, Hq, H = shape
    n, nq = 700, 3
    v = (_randn((n, H, D), 21) / 5).clamp(-1, 1) * 2.0 ** 126
    out = _run(_randn((n, H, D), 20), v, _randn((nq, Hq, D), 22), P, wide)
    assert torch.isfinite(out).all()
    # one token alone has all the weight of a row
    out = _run(_scored([0.0] * 40 + [90.0], H, D, 23), v[:41], torch.ones((1, Hq, D)), P, wide)
    assert torch.isfinite(out).all()
    # values in bfloat16's subnormals: the tolerance of their own last place
    tiny = (_randn((200, H, D), 24) * 2.0 ** -125).to(torch.bfloat16)
    k, q = _randn((200, H, D), 25).to(torch.bfloat16), _randn((1, Hq, D), 26).to(torch.bfloat16)
    cache = attn_kv4_cache(-(-200 // P), H, D, P)
    attn_kv4_append(k.cuda(), tiny.cuda(), _dev(range(200)), cache, P)
    table = _dev([list(range(cache.shape[0])) + [-1] * (80000 // P if wide else 0)])
    out, _ = attn_fwd_kv4(q.cuda(), _dev([0, 1]), _dev([200]), table, cache, P)
    (kc, ks, km), (vc, vs, vm) = ([x.transpose(1, 0, 2, 3).reshape(H, -1, x.shape[3])[:, :200] for x in side]
                                  for side in S.kv4_unpack(cache.cpu().numpy(), D, P))
    kv, vv = S.kv4_values(kc, ks, km), S.kv4_values(vc, vs, vm)
    for hq in range(Hq):
        h = hq // (Hq // H)
        x = D ** -0.5 * (kv[h] @ to_f64(q)[0, hq])
        p = np.exp(x - x.max())
        want = (p / p.sum()) @ vv[h]
        # one step of bfloat16 (its own half, and the sums' below that)
        assert (np.abs(to_f64(out)[0, hq] - want) <= 2.0 ** -133 + 2.0 ** -7 * np.abs(want)).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("power", [21, 27, 29, 36, 60])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (256, 64)])
def test_scores_past_float32s_whole_numbers(D, P, power, wide):
    # scores of about 2^power: one token has all the weight; float32 cannot hold a difference of ten beside them
    n = 90
    for at in (0, 50, 89):
        size = torch.linspace(0.5, 0.75, n)
        size[at] = 0.97
        k = (size * 2.0 ** (power - 10))[:, None, None] / math.sqrt(D) * torch.ones((n, 1, D))
        q = 2.0 ** 10 * torch.tensor([1.0, 0.9, -1.0])[None, :, None].expand(1, 3, D)
        v = _randn((n, 1, D), 27)
        out = _run(k, v, q, P, wide)
        # V's own codes: within half a scale, and bfloat16's half step
        near = (out[0, :2].float().cpu() - v[at].to(torch.bfloat16).float()).abs()
        assert (near <= 0.55 * (v[at].max() - v[at].min()) / 15 + 0.02).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (256, 64)])
def test_all_weight_on_tokens_without_a_scale(D, P, wide):
    # constant V (scale 0) has all the weight; the others' weights are 0 in float32, or nearly, however large their V is
    n = 100
    for low in (-150.0, -85.0, -40.0):
        scores = torch.where(torch.arange(n) % 3 == 0, 0.0, low)
        for power in (0, 20, 100):
            v = _randn((n, 1, D), 28) * 2.0 ** power
            v[::3] = 0.75
            _run(_scored(scores, 1, D, 29), v, torch.ones((2, 4, D)), P, wide)


@pytest.mark.parametrize("wide", [False, True])
def test_scales_that_spread_late(wide):
    # an item whose last tokens are the first to differ by more than 2^6: begun again, from tiles that were copied before
    for n, at in ((1000, 999), (1000, 500), (2500, 2400)):
        v = _randn((n, 2, 128), 30)
        v[at] *= 2.0 ** 9
        v[at - 1] *= 2.0 ** -30
        out = _run(_randn((n, 2, 128), 31), v, _randn((2, 8, 128), 32), 16, wide)
        assert torch.equal(out, _run(_randn((n, 2, 128), 31), v, _randn((2, 8, 128), 32), 16, wide))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_a_cache_made_by_hand_with_the_largest_scales(D, P, wide):
    # scales of 2^126 with codes 0 and 1: more than quantising gives, within what the layout and the ranges allow
    n, G = 50, D // 64
    pages = -(-n // P)
    cache = attn_kv4_cache(pages, 1, D, P)
    k = _randn((n, 1, D), 33).to(torch.bfloat16).cuda()
    attn_kv4_append(k, k, _dev(range(n)), cache, P)
    cache[:, :, 36 * G * P:68 * G * P] &= 0x11
    pairs = cache[:, :, 68 * G * P:].clone().view(torch.int16).view(pages, 1, G * P, 2)
    pairs[..., 0], pairs[..., 1] = 0x7E80, 0
    cache[:, :, 68 * G * P:] = pairs.view(torch.uint8).view(pages, 1, 4 * G * P)
    q = _randn((3, 4, D), 34).to(torch.bfloat16).cuda()
    table = _dev([list(range(pages)) + [-1] * (80000 // P if wide else 0)])
    out, lse = attn_fwd_kv4(q, _dev([0, 3]), _dev([n]), table, cache, P)
    assert attn_fwd_status() == 0 and torch.isfinite(out).all() and out.max() > 2.0 ** 122
    _check(out, lse, q, n, cache, D, P)
