"""The frequency table of rotary positions, entry by entry against exact
arithmetic on whole numbers (pi by the arithmetic-geometric mean)."""
import ctypes as C
import math
import random

import pytest

from test_abi import lib  # noqa: F401  (the built library)

BITS = 1500


def _pi():
    """floor(pi 2^BITS), by the Gauss-Legendre iteration."""
    n = BITS + 64
    one = 1 << n
    a, b, t, p = one, math.isqrt((one * one) >> 1), one >> 2, 1
    while abs(a - b) > 4:
        a, b, c = (a + b) >> 1, math.isqrt(a * b), a
        t -= p * ((c - a) ** 2) >> n
        p *= 2
    return ((a + b) ** 2 // (4 * t)) >> 64


PI = _pi()


def _exact(x):
    """x / (2 pi) modulo 1, times 2^64, to nearest."""
    n, d = x.as_integer_ratio()
    # n / d / (2 PI 2^-BITS) 2^64, rounded
    num, den = n << (BITS + 65), d * 2 * PI
    return ((num // den) + 1 >> 1) % (1 << 64)


def _table(lib, freqs):  # noqa: F811
    n = len(freqs)
    out = (C.c_longlong * (2 * n))()
    assert lib.attn_rope_table((C.c_double * n)(*freqs), (C.c_int * n)(*([0] * n)), n, 1, out) == 0
    return [v % (1 << 64) for v in out[0::2]]


def test_pi():
    assert str(PI * 10 ** 50 >> BITS) == "314159265358979323846264338327950288419716939937510"


@pytest.mark.parametrize("sign", [1, -1])
def test_rope_table_is_exact(lib, sign):  # noqa: F811
    r = random.Random(3)
    freqs = [10000.0 ** (-i / 64) for i in range(64)] + [6.5, 1000.3, 123456.7, 2 * math.pi, math.pi, 1e18, 1e300]
    freqs += [1.7976931348623157e308, 5e-324, 2.0 ** -64, 3e-19, 1e-12, 0.0]
    freqs += [math.ldexp(r.uniform(0.5, 1), r.randint(-70, 1024)) for _ in range(400)]
    freqs = [sign * f for f in freqs]
    got = _table(lib, freqs)
    for f, g in zip(freqs, got):
        off = (g - _exact(f)) % (1 << 64)
        assert off in (0, 1, (1 << 64) - 1), (f, g, _exact(f))  # (one step where the last place is in doubt)
    assert sum(g != _exact(f) for f, g in zip(freqs, got)) <= 2


def test_far_positions_of_large_frequencies(lib):  # noqa: F811
    # the angle of the farthest position, in turns: the table's rounding of 2^-65 times 2^31
    for f in (1.0, 6.5, 1000.3, 123456.7, 1e9):
        t = _table(lib, [f])[0]
        for pos in (2 ** 31 - 1, -2 ** 31, 1234567891):
            n, d = f.as_integer_ratio()
            exact = ((n * pos << (BITS + 64)) // (d * 2 * PI)) % (1 << 64)
            off = (t * pos - exact) % (1 << 64)
            assert min(off, (1 << 64) - off) <= 2 ** 30 + 1, (f, pos)


@pytest.mark.gpu
def test_far_positions_of_large_frequencies_on_the_gpu():
    # angles reduced in whole numbers; y within 2^-20 (|x1| + |x2|) before its rounding to bfloat16 (test_gpu_rope)
    import torch

    from exact_attention_attn_gb300 import attn_rope, attn_rope_table
    D = 64
    inv = [1.0, 6.5, 1000.3, 123456.7, -1e9, 1e300, 0.3] + [1.7 ** i for i in range(25)]
    pos = [2 ** 31 - 1, -2 ** 31, 1234567891, 7, 0]
    x = torch.randn((1, 2, len(pos), D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    y, _ = attn_rope(x, None, torch.tensor([[pos]], dtype=torch.int32).cuda(), attn_rope_table(D, inv_freq=inv))
    x, y = x.double().cpu(), y.double().cpu()
    for i, f in enumerate(inv):
        n, d = f.as_integer_ratio()
        for t, p in enumerate(pos):
            turns = ((n * p << (BITS + 64)) // (d * 2 * PI)) % (1 << 64) / 2.0 ** 64
            c, s = math.cos(2 * math.pi * turns), math.sin(2 * math.pi * turns)
            a, b = x[0, :, t, i], x[0, :, t, i + 32]
            for got, want in ((y[0, :, t, i], a * c - b * s), (y[0, :, t, i + 32], b * c + a * s)):
                assert ((got - want).abs() <= 2.0 ** -20 * (a.abs() + b.abs()) + 2.0 ** -8 * want.abs()).all(), (f, p)
