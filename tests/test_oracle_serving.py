"""Pins of oracle/serving.py: rotary positions, pages, the 4-bit cache and
attention over it, against closed forms, torch and invariants; planted mistakes
are caught."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S


def test_to_bf16_matches_torch():
    r = np.random.default_rng(0)
    x = (r.standard_normal(20000) * np.exp(r.uniform(-40, 40, 20000))).astype(np.float32)
    ties = (np.arange(1, 2000, dtype=np.uint32) << 16 | 0x8000).view(np.float32)
    x = np.concatenate([x, ties, -ties, [0.0, 1.0, 255.5]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(S.to_bf16(x.astype(np.float64)), want)


def _rope_case(adjacent, seed=1):
    r = np.random.default_rng(seed)
    x = r.standard_normal((2, 3, 5, 16))
    pos = r.integers(0, 1000, (3, 2, 5))
    inv = 100.0 ** (-np.arange(6) / 6.0)
    return x, pos, inv, [0, 1, 2, 0, 1, 1]


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_is_complex_multiplication_and_its_gradient(adjacent):
    x, pos, inv, axis = _rope_case(adjacent)
    y = S.rope(x, pos, inv, axis, adjacent)
    a, b = (x[..., 0:12:2], x[..., 1:12:2]) if adjacent else (x[..., :6], x[..., 6:12])
    phi = np.stack([pos[a_] * f for a_, f in zip(axis, inv)], -1)[:, None]
    z = (a + 1j * b) * np.exp(1j * phi)
    got = y[..., 0:12:2] + 1j * y[..., 1:12:2] if adjacent else y[..., :6] + 1j * y[..., 6:12]
    assert np.abs(z - got).max() < 1e-12
    assert np.array_equal(y[..., 12:], x[..., 12:])
    # lengths are kept, position 0 is the identity, the backward undoes the forward
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    assert np.array_equal(S.rope(x, 0 * pos, inv, axis, adjacent), x)
    assert np.allclose(S.rope(y, pos, inv, axis, adjacent, backward=True), x)
    # gradient of sum(w * y) by autograd of the complex form, and by differences
    w = np.random.default_rng(3).standard_normal(x.shape)
    dx = S.rope(w, pos, inv, axis, adjacent, backward=True)
    for i in [(0, 0, 0, 0), (1, 2, 4, 7), (0, 1, 3, 11), (1, 0, 2, 14)]:
        e = np.zeros_like(x)
        e[i] = 1e-3
        d = ((S.rope(x + e, pos, inv, axis, adjacent) - S.rope(x - e, pos, inv, axis, adjacent)) * w).sum() / 2e-3
        assert abs(d - dx[i]) < 1e-9
    # only differences of positions matter to q . k
    q, k = S.rope(x, pos, inv, axis, adjacent), S.rope(x[::-1], pos, inv, axis, adjacent)
    q2, k2 = S.rope(x, pos + 77, inv, axis, adjacent), S.rope(x[::-1], pos + 77, inv, axis, adjacent)
    assert np.allclose((q * k).sum(-1), (q2 * k2).sum(-1))


def test_rope_planted_mistakes():
    x, pos, inv, axis = _rope_case(False)
    y = S.rope(x, pos, inv, axis)
    assert not np.allclose(y, S.rope(x, pos, inv, [0] * 6))
    assert not np.allclose(y, S.rope(x, pos, inv, axis, adjacent=True))
    assert not np.allclose(y, S.rope(x, pos, inv, axis, backward=True))
    assert not np.allclose(y, S.rope(x, pos, 1 / inv, axis))


def test_pages_by_hand():
    table = np.full((3, 4), -1)
    table[0, :2] = [7, 3]
    free = np.array([10, 11, 12, 13, 14, 0, 0])
    got = S.pages_assign(table, [20, 0, 16], [1, 33, 0], free, 5, 16, 40)
    assert got["info"] == [0, 34] and got["free_count"] == 2
    assert got["table"].tolist() == [[7, 3, -1, -1], [14, 13, 12, -1], [-1, -1, -1, -1]]
    assert got["cu"].tolist() == [0, 1, 34, 34] and got["lens"].tolist() == [21, 33, 16]
    assert got["slots"][:3].tolist() == [3 * 16 + 4, 14 * 16, 14 * 16 + 1] and got["slots"][33] == 12 * 16
    assert got["slots"][34:].tolist() == [-1] * 6 and got["positions"][:2].tolist() == [20, 0]
    back = S.pages_release(got["table"], got["lens"], [-1, 17, 50], free, 2, 16)
    assert back["info"] == [0, 1] and back["free"][2] == 12 and back["lens"].tolist() == [21, 17, 16]
    assert back["table"][1].tolist() == [14, 13, -1, -1]
    for new, count, most, bit in (([65, 0, 0], 5, 99, 1), ([1, 33, 0], 5, 33, 2), ([1, 33, 0], 2, 40, 4), ([0, 0, 0], 8, 40, 8)):
        bad = S.pages_assign(table, [0, 0, 16], new, free, count, 16, most)
        assert bad["info"] == [bit, 0] and np.array_equal(bad["table"], table) and (bad["slots"] == -1).all()


def test_pages_without_a_slot():
    # page 2^27 of 16 tokens would have slot 2^31; -1 is no page
    free = np.array([2 ** 27, -1, 2 ** 27 - 1])
    got = S.pages_assign(np.full((1, 3), -1), [0], [33], free, 3, 16, 33)
    assert got["info"] == [0, 33] and got["table"].tolist() == [[2 ** 27 - 1, -1, 2 ** 27]]
    assert got["slots"].tolist() == list(range(2 ** 31 - 16, 2 ** 31)) + [-2] * 17


def test_kv4_quantise():
    r = np.random.default_rng(5)
    x = S.to_bf16(r.standard_normal((7, 3, 192)) * np.exp(r.uniform(-3, 3, (7, 3, 192))))
    c, s, m, q = S.kv4_quantise(x)
    v = S.kv4_values(c, s, m)
    step = np.repeat(s, 64, -1).reshape(x.shape)
    # half a step, and 15 times the scale's own rounding (2^-8) at the top of the range
    assert (np.abs(v - x) <= step * (0.5 + 15 * 2.0 ** -8)).all()
    y = x.reshape(7, 3, 3, 64)
    assert np.array_equal(m, y.min(-1)) and c.min() == 0 and c.max() == 15
    # a straight line of 16 values is held exactly
    line = np.tile(np.arange(16.0) * 0.25 - 1, 4)
    c, s, m, _ = S.kv4_quantise(line)
    assert s == 0.25 and m == -1 and np.array_equal(S.kv4_values(c, s, m), line)
    # (max - m) / 15 = 2.2890625 and 2.4140625, halfway between two bfloat16 numbers
    for hi, lo, want in ((1.8359375, -32.5, 2.296875), (34.25, -1.9609375, 2.421875)):
        x = np.full(64, lo)
        x[3] = hi
        c, s, m, q = S.kv4_quantise(x)
        assert s == want and m == lo and c[3] == 15 and c[4] == 0 and q[3] == (hi - lo) / want
    c, s, m, _ = S.kv4_quantise(np.full(64, 3.5))
    assert s == 0 and (c == 0).all() and m == 3.5


def test_kv4_unpack_and_attention():
    r = np.random.default_rng(6)
    D, P, H = 128, 16, 2
    cache = np.zeros((3, H, 72 * 2 * P), dtype=np.uint8)
    # token 5, head 1, K dim 64 + 6 = 9; its pair (2.0, -1.5); by the byte offsets of the definition
    cache[2, 1, (1 * P + 5) * 32 + 3] = 9
    cache[2, 1, (1 * P + 5) * 32 + 4] = 11 << 4
    at = 32 * 2 * P + (1 * P + 5) * 4
    cache[2, 1, at:at + 4] = np.array([0x4000, 0xBFC0], dtype=np.uint16).view(np.uint8)
    (ck, sk, mk), (cv, sv, mv) = S.kv4_unpack(cache, D, P)
    k = S.kv4_values(ck, sk, mk)
    assert k[2, 1, 5, 70] == 9 * 2.0 - 1.5 and k[2, 1, 5, 73] == 11 * 2.0 - 1.5 and k[2, 1, 5, 64] == -1.5
    assert k[2, 1, 5, :64].any() == False and S.kv4_values(cv, sv, mv).any() == False  # noqa: E712
    # paged attention equals attention on the gathered rows; order of pages, lengths and empty requests matter
    k, v = r.standard_normal((6, H, P, D)), r.standard_normal((6, H, P, D))
    q = r.standard_normal((5, 4, D))
    table, lens, cu = np.array([[4, 1, -1], [0, -1, -1], [5, 2, 3]]), [20, 0, 33], [0, 1, 2, 5]
    O, L = S.attention_requests(q, cu, lens, table, k, v, P, 0.1, True)
    want, wl = oracle.attention_bruteforce(q[2:5].transpose(1, 0, 2)[None],
                                           np.concatenate([k[5], k[2], k[3]], 1)[None, :, :33],
                                           np.concatenate([v[5], v[2], v[3]], 1)[None, :, :33], 0.1, True)
    assert np.allclose(O[2:5], want[0].transpose(1, 0, 2)) and np.allclose(L[2:5], wl[0].T)
    assert (O[1] == 0).all() and np.isneginf(L[1]).all()
    assert not np.allclose(S.attention_requests(q, cu, lens, table[:, ::-1], k, v, P, 0.1, True)[0][2:5], O[2:5])
    assert math.isclose(L[0, 0], float(torch.logsumexp(torch.from_numpy(
        np.concatenate([k[4, 0], k[1, 0]])[:20] @ q[0, 0] * 0.1), 0)))


def test_kv4_scale_is_the_quotient_by_fifteen():
    # against exact fractions: the nearest bfloat16 number, and at a tie (or within float32's reach of one) a neighbour
    from fractions import Fraction
    r = np.random.default_rng(21)
    lo = S.to_bf16(-np.exp2(r.uniform(-130, 120, 4000)))
    hi = S.to_bf16(-lo * np.exp2(r.uniform(-9, 9, 4000)))
    for hi_, lo_ in ((1.8359375, -32.5), (34.25, -1.9609375), (34.0, -0.3359375), (2.28125 * 15 - 1, -1.0)):
        hi, lo = np.append(hi, hi_), np.append(lo, lo_)
    s, ties = S.kv4_scale(lo, hi), 0
    for m, h, got in zip(lo, hi, s):
        exact = (Fraction(float(h)) - Fraction(float(m))) / 15
        step = Fraction(2) ** max(math.frexp(float(exact))[1] - 8, -133)
        off = abs(Fraction(float(got)) - exact) / step
        ties += off == Fraction(1, 2)
        assert off <= Fraction(1, 2) + Fraction(1, 2 ** 13), (m, h, got)
    assert ties >= 3


def test_planted_mistakes_in_the_scale_are_seen():
    # another factor, or a quotient that is cut instead of rounded, does not agree with the quotient by 15 (a factor
    # nearer than some 2^-13 would: spans of 9 bits over 15 lie no closer to a tie)
    r = np.random.default_rng(22)
    x = S.to_bf16(r.standard_normal((200, 64)))
    m, hi = x.min(-1), x.max(-1)
    good = S.kv4_scale(m, hi)
    for wrong in (np.float32(1.06), np.float32(17 / 16), np.float32(1.0)):
        assert (S.to_bf16((hi - m) / 16 * float(wrong)) != good).any()
    bits = ((hi - m) / 15).astype(np.float32).view(np.uint32) & np.uint32(0xffff0000)
    assert (bits.view(np.float32) != good).any()
