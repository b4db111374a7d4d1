"""The 4-bit cache and attention over it, against the float64 oracle.

Codes, scales and minima are compared exactly: the oracle's scale is the bfloat16
number nearest to the float64 quotient by 15, and where that is within float32's
reach of a tie the one that the format's float32 product goes to; a code may
differ only where the exact quotient is within 2^-19 of a tie (the float32
difference x - m and the quotient are each off by at most 2^-24 of a value up to
15, twice).

Attention tolerance, per element, from the arithmetic:
  scores  float32 accumulation of exact products: at most 16 roundings (a tensor
          core's step may cut instead of round, 2^-23) of partial sums that are
          at most Sabs = scale sum_d |q_d| (s c + |m|), in log2 units another
          few: dS = 2^-18 max_j Sabs
  weights exp2 2^-22 relative, the weight rounded to half precision 2^-11
  output  float32 sums (2^-20 of the absolute sum), one rounding to bfloat16 2^-8
so |dO| <= (2^-11 + 2 dS + 2^-19) A + 2^-8 |O|, A = softmax-weighted sum of s c + |m|,
and |dLSE| <= dS + 2^-20 (1 + |LSE|).  (A weight times scale in
half precision's subnormals is off by 2^-25 at most, where the largest scale is in
[1/2, 1) and the largest weight at least 2^10: with scales that differ by a factor
of 2 at the heavy tokens, as here, 2^-33 of the products' sum each, for n <= 2^14
tokens 2^-19 of it.  Caches whose scales differ by more are test_gpu_kv4_ranges'.)"""
import math

import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import (AttnError, attn_fwd, attn_fwd_kv4, attn_fwd_status, attn_kv4_append,
                                        attn_kv4_cache, attn_kv4_page_bytes, attn_kv4_read)
from exact_attention_attn_gb300.workloads import to_f64
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _randn(shape, seed, amp=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * amp).to(torch.bfloat16).cuda()


# ---------------------------------------------------------------- append and read

def _check_codes(x, slots, cache, D, P, side):
    """The cache's rows of the slots against the quantisation of x [T, H, D] (float64)."""
    c, s, m, q = S.kv4_quantise(x)
    gc, gs, gm = S.kv4_unpack(cache.cpu().numpy(), D, P)[side]
    t = np.flatnonzero(slots >= 0)
    page, off = slots[t] // P, slots[t] % P
    assert np.array_equal(gs[page, :, off], s[t]) and np.array_equal(gm[page, :, off], m[t])
    differ = gc[page, :, off] != c[t]
    frac = np.abs(q[t] - np.floor(q[t]) - 0.5)
    assert (frac[differ] < 2.0 ** -19).all(), (differ.sum(), frac[differ])
    return S.kv4_values(gc, gs, gm)


@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (33, 2, 128, 16), (5, 8, 128, 64), (777, 3, 192, 32), (64, 1, 1024, 16),
                                     (1000, 4, 256, 64), (31, 16, 64, 32)])
def test_append_then_read(T, H, D, P):
    pages = -(-T // P) + 3
    r = np.random.default_rng(T)
    slots = r.permutation(pages * P)[:T]
    slots[r.random(T) < 0.1] = -1
    k, v = _randn((T, H, D), T), _randn((T, H, D), T + 1, 20.0)
    cache = attn_kv4_cache(pages, H, D, P)
    cache.fill_(0xA5)
    before = cache.cpu().numpy().copy()
    d_slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
    attn_kv4_append(k, v, d_slots, cache, P)
    kv = _check_codes(to_f64(k), slots, cache, D, P, 0)
    vv = _check_codes(to_f64(v), slots, cache, D, P, 1)
    # nothing else was written
    G, held = D // 64, np.zeros((pages, P), dtype=bool)
    held.reshape(-1)[slots[slots >= 0]] = True
    after = cache.cpu().numpy()
    for at, n in ((0, 32), (32 * G * P, 4), (36 * G * P, 32), (68 * G * P, 4)):
        a, b = (z[:, :, at:at + n * G * P].reshape(pages, H, G, P, n) for z in (after, before))
        assert np.array_equal(a.transpose(0, 3, 1, 2, 4)[~held], b.transpose(0, 3, 1, 2, 4)[~held])
    ok, ov = attn_kv4_read(d_slots, cache, P)
    for got, val in ((ok, kv), (ov, vv)):
        want = np.where((slots >= 0)[:, None, None], val[slots // P, :, slots % P], 0.0).transpose(1, 0, 2)
        # s c + m in float32 (2^-24 of the result), then bfloat16's half step
        assert (np.abs(to_f64(got) - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
    assert attn_fwd_status() == 0


def test_append_strides_and_read_into_views():
    T, H, D, P = 37, 3, 128, 32
    qkv = _randn((T, 3 * H, D), 5)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(0))[:T].to(torch.int32).cuda()
    a, b = attn_kv4_cache(2, H, D, P), attn_kv4_cache(2, H, D, P)
    attn_kv4_append(k, v, slots, a, P)
    attn_kv4_append(k.contiguous(), v.contiguous(), slots, b, P)
    assert torch.equal(a, b)
    c = attn_kv4_cache(2, H, D, P)
    heads_first = k.transpose(0, 1).contiguous().transpose(0, 1)
    attn_kv4_append(heads_first, v, slots, c, P)
    assert torch.equal(a, c)
    ok, ov = attn_kv4_read(slots, a, P)
    room = torch.zeros((T, H, 2 * D), dtype=torch.bfloat16, device="cuda")
    vk, vv = room[..., :D].transpose(0, 1), room[..., D:].transpose(0, 1)
    attn_kv4_read(slots, a, P, out_k=vk, out_v=vv)
    assert torch.equal(vk, ok) and torch.equal(vv, ov)


def test_special_groups():
    D, P = 128, 16
    x = torch.zeros((9, 1, D), dtype=torch.bfloat16)
    x[0] = 3.0                                     # constant: scale 0
    x[1, 0, :64] = torch.arange(64) % 16           # exact
    x[2, 0, 5] = float("inf")
    x[3, 0, 70] = float("nan")
    x[4, 0, 1], x[4, 0, 2] = 3.3e38, -3.3e38       # spread past float32's largest value
    x[5, 0, :64] = torch.tensor([2.0 ** -133 * (i % 3) for i in range(64)])   # subnormal
    x[6, 0, 0] = -float("inf")
    x[7, 0, :64] = torch.linspace(-1e-38, 2e-38, 64)
    x[8, 0, :64] = torch.linspace(-1, 1, 64)
    slots = torch.arange(9, dtype=torch.int32).cuda()
    cache = attn_kv4_cache(1, 1, D, P)
    attn_kv4_append(x.cuda(), x.cuda(), slots, cache, P)
    (c, s, m), (c2, s2, m2) = S.kv4_unpack(cache.cpu().numpy(), D, P)
    assert np.array_equal(c, c2) and np.array_equal(s, s2, equal_nan=True) and np.array_equal(m, m2, equal_nan=True)
    c, s, m = c[0, 0], s[0, 0], m[0, 0]
    for t, g in ((2, 0), (3, 1), (6, 0)):
        assert np.isnan(s[t, g]) and np.isnan(m[t, g]) and (c[t, g * 64:g * 64 + 64] == 0).all()
        assert s[t, 1 - g] == 0 and m[t, 1 - g] == 0
    wc, ws, wm, q = S.kv4_quantise(x.double().numpy()[[0, 1, 4, 5, 7, 8], 0])
    rows = [0, 1, 4, 5, 7, 8]
    assert np.array_equal(s[rows], ws) and np.array_equal(m[rows], wm)
    differ = c[rows] != wc
    assert (np.abs(q - np.floor(q) - 0.5)[differ] < 2.0 ** -19).all()
    ok, _ = attn_kv4_read(slots, cache, P)
    assert torch.equal(ok[0, 1, :64].cpu(), x[1, 0, :64]) and torch.isnan(ok[0, 2, :64]).all() and (ok[0, 0] == 3).all()


def test_scales_halfway_between_two_numbers():
    # groups with one large value: their (max - min) / 15 often lies halfway between two bfloat16 numbers
    T, H, D, P = 4096, 2, 64, 16
    g = torch.Generator().manual_seed(11)
    x = torch.rand((T, H, D), generator=g) * 2 - 1
    x[..., 0] = 1 + 3 * torch.rand((T, H), generator=g)
    x[..., 1] = -(32 + 40 * torch.rand((T, H), generator=g))
    x = torch.where(torch.rand((T, H, 1), generator=g) < 0.5, x, -x).to(torch.bfloat16)
    span = (x.double().amax(-1) - x.double().amin(-1)) / 15
    low = torch.tensor(S.to_bf16(span.numpy() * (1 - 2.0 ** -20)))
    high = torch.tensor(S.to_bf16(span.numpy() * (1 + 2.0 ** -20)))
    assert ((low + high) / 2 == span)[low != high].sum() > 20  # the inputs hold such groups
    cache, slots = attn_kv4_cache(T // P, H, D, P), np.arange(T)
    attn_kv4_append(x.cuda(), (-x).cuda(), torch.tensor(slots, dtype=torch.int32, device="cuda"), cache, P)
    _check_codes(x.double().numpy(), slots, cache, D, P, 0)
    _check_codes(-x.double().numpy(), slots, cache, D, P, 1)


def test_bad_slots_are_skipped_and_reported():
    T, H, D, P = 6, 2, 64, 16
    k = _randn((T, H, D), 1)
    cache = attn_kv4_cache(2, H, D, P)
    slots = torch.tensor([0, 32, -2, 2 ** 31 - 1, -(2 ** 31), 5], dtype=torch.int32).cuda()
    attn_kv4_append(k, k, slots, cache, P)
    assert attn_fwd_status() == -7 and attn_fwd_status() == 0
    good = attn_kv4_cache(2, H, D, P)
    pick = torch.tensor([0, 5], device="cuda")
    attn_kv4_append(k[pick], k[pick], slots[pick], good, P)
    assert torch.equal(cache, good)
    ok, ov = attn_kv4_read(slots, cache, P)
    assert attn_fwd_status() == -7
    assert (ok[:, 1:5] == 0).all() and (ov[:, 1:5] == 0).all() and (ok[:, 0] != 0).any()
    assert attn_fwd_status() == 0
    empty = attn_kv4_cache(0, H, D, P)
    attn_kv4_append(k, k, torch.full((T,), -1, dtype=torch.int32, device="cuda"), empty, P)
    assert attn_fwd_status() == 0


# ---------------------------------------------------------------- attention

def _random_cache(pages, H, D, P, seed, v_amp=1.0):
    """A full cache of random pages, and its values (float64)."""
    T = pages * P
    cache = attn_kv4_cache(pages, H, D, P)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    attn_kv4_append(_randn((T, H, D), seed), _randn((T, H, D), seed + 1, v_amp), slots, cache, P)
    return cache


def _values(cache, D, P):
    k, v = S.kv4_unpack(cache.cpu().numpy(), D, P)
    size = lambda c, s, m: S.kv4_values(c, s, np.abs(m))  # noqa: E731
    return S.kv4_values(*k), S.kv4_values(*v), size(*k), size(*v)


def _check_attention(out, lse, q, cu, lens, table, cache, D, P, scale, causal):
    k, v, ka, va = _values(cache, D, P)
    qf = to_f64(q)
    O, L = S.attention_requests(qf, cu, lens, table, k, v, P, scale, causal)
    got, gl = to_f64(out), to_f64(lse)
    group = q.shape[1] // cache.shape[1]
    for r in range(len(lens)):
        a, b, n = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if b == a:
            continue
        ids = [int(i) for i in table[r][:-(-n // P)]]
        flat = lambda x: x[ids].transpose(1, 0, 2, 3).reshape(x.shape[1], -1, D)[:, :n]  # noqa: E731
        kr, kar, var = flat(k), flat(ka), flat(va)
        for t in range(a, b):
            seen = min(n, max(0, t - a + 1 + n - (b - a))) if causal else n
            for h in range(q.shape[1]):
                kv = h // group
                if seen == 0:
                    assert (got[t, h] == 0).all() and np.isneginf(gl[t, h])
                    continue
                x = scale * kr[kv, :seen] @ qf[t, h]
                big = abs(scale) * (kar[kv, :seen] @ np.abs(qf[t, h])).max()
                p = np.exp(x - L[t, h])
                A = p @ var[kv, :seen]
                dS = 2.0 ** -18 * big
                tol = (2.0 ** -11 + 2 * dS + 2.0 ** -19) * A + 2.0 ** -8 * np.abs(O[t, h])
                err = np.abs(got[t, h] - O[t, h])
                assert (err <= tol).all(), (r, t, h, (err / tol).max())
                assert abs(gl[t, h] - L[t, h]) <= dS + 2.0 ** -20 * (1 + abs(L[t, h])), (r, t, h, gl[t, h], L[t, h])


def _requests(lens, nq, P, width, pages, seed):
    r = np.random.default_rng(seed)
    ids = r.permutation(pages)
    table, at = np.full((len(lens), width), -1), 0
    for i, n in enumerate(lens):
        c = -(-n // P)
        table[i, :c] = ids[at:at + c]
        at += c
    return table, np.concatenate([[0], np.cumsum(nq)])


def _run(lens, nq, Hq, H, D, P, causal=True, scale=None, seed=0, width=None, v_amp=1.0, pad=0, q_amp=1.0):
    need = sum(-(-n // P) for n in lens)
    cache = _random_cache(max(1, need), H, D, P, seed, v_amp)
    width = max(1, max(-(-n // P) for n in lens)) if width is None else width
    table, cu = _requests(lens, nq, P, width, need, seed)
    T = int(cu[-1]) + pad
    q = _randn((T, Hq, D), seed + 7, q_amp)
    # whatever the pages hold past a request's end must not matter
    raw = cache.view(cache.shape[0], H, -1)
    G = D // 64
    for i, n in enumerate(lens):
        if n % P:
            page = int(table[i, n // P])
            for at, w in ((0, 32), (32 * G * P, 4), (36 * G * P, 32), (68 * G * P, 4)):
                raw[page, :, at:at + w * G * P].view(H, G, P, w)[:, :, n % P:] = 0xFF  # NaN pairs
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float32, device="cuda")
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    attn_fwd_kv4(q, dev(cu), dev(lens), dev(table), cache, P, scale=scale, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    assert attn_fwd_status() == 0
    _check_attention(out, lse, q, cu, lens, table, cache, D, P, scale, causal)
    if pad:  # rows behind the last request are left as they were
        assert torch.isnan(out[-pad:]).all() and torch.isnan(lse[-pad:]).all()
    return out, lse


CASES = [
    # lens, query tokens, Hq, Hkv, D, P
    ((1,), (1,), 1, 1, 64, 16),
    ((16,), (1,), 4, 1, 64, 16),
    ((17,), (1,), 8, 1, 128, 16),
    ((63, 64, 65, 1), (1, 1, 1, 1), 8, 2, 128, 64),
    ((129, 300, 5), (1, 1, 1), 32, 8, 128, 32),
    ((1000, 0, 77), (1, 1, 1), 6, 2, 192, 16),
    ((640, 511), (1, 1), 16, 2, 256, 64),
    ((200, 31, 90), (4, 1, 7), 8, 2, 128, 16),
    ((200, 31, 90), (4, 0, 9), 12, 4, 64, 32),
    ((100, 64), (33, 64), 10, 2, 128, 16),
    ((330, 64, 0, 200), (33, 50, 1, 40), 8, 2, 64, 32),
    ((500, 77), (40, 70), 8, 2, 128, 64),
    ((70, 40), (5, 3), 16, 1, 256, 16),
    ((5, 3), (9, 3), 4, 2, 64, 16),          # more query tokens than keys: rows that see none
    ((2500,), (1,), 64, 1, 128, 16),
    ((300,) * 40, (1,) * 40, 4, 4, 64, 16),
    ((4096,), (2,), 8, 8, 64, 64),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}q{max(c[1])}h{c[2]}k{c[3]}d{c[4]}p{c[5]}")
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_oracle(case, causal):
    lens, nq, Hq, H, D, P = case
    _run(list(lens), list(nq), Hq, H, D, P, causal=causal, seed=sum(lens) + D)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}q{max(c[1])}h{c[2]}k{c[3]}d{c[4]}p{c[5]}")
def test_attention_under_a_table_for_long_contexts(case):
    # items cut into pieces and merged by the second kernel, whatever the lengths
    _run(*map(list, case[:2]), *case[2:], width=80000 // case[5], pad=2)


@pytest.mark.parametrize("lens,nq,Hq,H,D,P,width", [
    ((2900,), (1,), 8, 1, 128, 16, None), ((2900,), (1,), 8, 1, 128, 16, 800), ((7000,), (2,), 3, 1, 64, 32, None),
    ((33, 0, 5), (1, 1, 1), 8, 2, 128, 16, 150), ((1, 2000, 0, 700), (1, 1, 0, 2), 4, 2, 64, 16, None),
    ((1800, 40), (1, 5), 4, 1, 192, 16, None), ((3500,), (1,), 4, 2, 256, 64, None), ((900, 1500), (5, 3), 8, 2, 256, 32, None),
    ((1500, 900), (70, 66), 4, 1, 64, 16, None), ((1500, 900), (70, 20), 4, 1, 128, 64, None), ((9000,), (1,), 5, 1, 128, 64, None),
    ((1200,) * 9, (1,) * 9, 16, 4, 128, 16, None)], ids=str)
def test_items_spread_over_a_cluster(lens, nq, Hq, H, D, P, width):
    _run(list(lens), list(nq), Hq, H, D, P, seed=len(lens) + D, width=width, pad=1)


def test_a_cluster_gives_the_same_bits_every_time():
    H, D, P = 2, 128, 16
    cache = _random_cache(200, H, D, P, 7)
    q = _randn((3, 8, D), 8)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q, dev([0, 1, 2, 3]), dev([3100, 900, 17]), dev([list(range(200))] * 3), cache, P)
    o, lse = attn_fwd_kv4(*args)
    for _ in range(20):
        a, b = attn_fwd_kv4(*args)
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
def test_attention_scales(scale):
    _run([150, 33], [1, 2], 8, 2, 128, 16, scale=scale, seed=3)


@pytest.mark.parametrize("v_amp,q_amp", [(1e-30, 1.0), (1e30, 1e-20), (1.0, 1e-30), (300.0, 30.0)])
def test_attention_ranges(v_amp, q_amp):
    # values and queries far from one: the powers of two that half precision is kept in range by
    _run([150, 40], [1, 1], 8, 2, 128, 16, seed=5, v_amp=v_amp, q_amp=q_amp)


def test_attention_wide_table_and_padding():
    _run([90, 4, 33], [1, 1, 2], 8, 2, 128, 16, seed=6, width=500, pad=5)


def test_attention_growing_scores_and_scales():
    # the largest score and the largest V come last, so that every reference has to move
    H, D, P, n = 1, 128, 16, 400
    k, v = _randn((n, H, D), 1), _randn((n, H, D), 2)
    ramp = torch.linspace(0, 12, n, device="cuda")[:, None, None]
    k = (k * 0.05 + ramp / 8).to(torch.bfloat16)
    v = (v * torch.exp(3 * ramp - 20)).to(torch.bfloat16)
    cache = attn_kv4_cache(25, H, D, P)
    attn_kv4_append(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), cache, P)
    q = torch.ones((1, 4, D), dtype=torch.bfloat16, device="cuda") * torch.tensor([1, -1, 0.1, 0], device="cuda")[None, :, None]
    q = q.to(torch.bfloat16)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = [list(range(25))]
    out, lse = attn_fwd_kv4(q, dev([0, 1]), dev([n]), dev(table), cache, P)
    _check_attention(out, lse, q, [0, 1], [n], table, cache, D, P, D ** -0.5, True)


def test_nan_reaches_only_rows_that_see_it():
    H, D, P, n, nq = 2, 128, 16, 90, 4
    k, v = _randn((n, H, D), 1), _randn((n, H, D), 2)
    v[n - 2, 0, 3] = float("nan")      # visible to the last two query tokens' rows of kv head 0
    k[n - 1, 1, 100] = float("inf")    # to the last query token's rows of kv head 1
    cache = attn_kv4_cache(6, H, D, P)
    attn_kv4_append(k, v, torch.arange(n, dtype=torch.int32, device="cuda"), cache, P)
    q = _randn((nq, 4, D), 3)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = attn_fwd_kv4(q, dev([0, nq]), dev([n]), dev([list(range(6))]), cache, P)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[2:, :2, :64] = True           # the poisoned group of V alone
    want[3:, 2:] = True
    assert torch.equal(nan, want)
    assert torch.equal(torch.isnan(lse), want[..., 100])
    q[0, 1, 7] = float("nan")
    out2, _ = attn_fwd_kv4(q, dev([0, nq]), dev([n]), dev([list(range(6))]), cache, P)
    want[0, 1] = True
    assert torch.equal(torch.isnan(out2), want) and torch.equal(out2[1, 3], out[1, 3])


def test_deterministic_and_shared_pages():
    # the same request twice, sharing its pages, gives the same bits in one call and in two
    H, D, P, n = 2, 128, 32, 5000
    cache = _random_cache(-(-n // P), H, D, P, 4)
    q = _randn((1, 8, D), 8).expand(2, 8, D).contiguous()
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = dev([list(range(-(-n // P)))] * 2)
    args = (q, dev([0, 1, 2]), dev([n, n]), table, cache, P)
    a, la = attn_fwd_kv4(*args)
    b, lb = attn_fwd_kv4(*args)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert (a[0].float() - a[1].float()).abs().max() <= 2.0 ** -7 * a.float().abs().max()


def test_bad_metadata_is_reported_and_stays_in_range():
    H, D, P = 2, 64, 16
    cache = _random_cache(4, H, D, P, 4)
    q = _randn((3, 4, D), 8)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(cu=[0, 1, 2], lens=[30, 40], table=[[0, 1, 3], [2, 3, 1]])
    ref, _ = attn_fwd_kv4(q, *(dev(good[n]) for n in ("cu", "lens", "table")), cache, P)
    assert attn_fwd_status() == 0
    for bad in (dict(table=[[0, 1, 3], [2, 99, 1]]), dict(table=[[0, 1, 3], [2, -1, 1]]), dict(lens=[30, 1000]),
                dict(lens=[30, -4]), dict(cu=[0, 1, 77]), dict(cu=[0, 1, -5]), dict(lens=[30, 2 ** 31 - 1])):
        a = {**good, **bad}
        out, _ = attn_fwd_kv4(q, dev(a["cu"]), dev(a["lens"]), dev(a["table"]), cache, P)
        assert attn_fwd_status() == -7, bad
        assert torch.allclose(out[0].float(), ref[0].float(), rtol=2.0 ** -6, atol=1e-4), bad  # the other request stands
    assert attn_fwd_status() == 0


@pytest.mark.parametrize("B", [3, 40, 300])
def test_descending_cu_is_reported_and_costs_no_work(B):
    # each other request would claim all the tokens: B / 2 times the work that the sizes allow
    H, D, P, T = 2, 64, 16, 1024
    cache = _random_cache(8, H, D, P, 4)
    q = _randn((T, 4, D), 8)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, lens = [T * (i & 1) for i in range(B + 1)], dev([128] * B)
    table = dev([list(range(8))] * B)
    out, lse = torch.full((T, 4, D), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, 4), 5.0, device="cuda")
    attn_fwd_kv4(q, dev(cu), lens, table, cache, P, out=out, lse=lse)
    assert attn_fwd_status() == -7
    assert (out == 5).all() and (lse == 5).all()
    cu = [0] * (B - 1) + [T, T]
    attn_fwd_kv4(q, dev(cu), lens, table, cache, P, causal=False, out=out, lse=lse)
    assert attn_fwd_status() == 0 and torch.isfinite(lse).all() and (lse[:, 0] != 5).any()


def test_no_pages_and_no_tokens():
    H, D, P = 1, 64, 16
    q = _randn((2, 2, D), 1)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = attn_kv4_cache(0, H, D, P)
    out, lse = attn_fwd_kv4(q, dev([0, 2]), dev([0]), torch.zeros((1, 0), dtype=torch.int32, device="cuda"), empty, P)
    assert attn_fwd_status() == 0 and (out == 0).all() and torch.isneginf(lse).all()
    out, lse = attn_fwd_kv4(q, dev([0]), dev([]), torch.zeros((0, 3), dtype=torch.int32, device="cuda"), empty, P)
    assert out.shape == q.shape


def test_refusals_on_the_device_side():
    cache = attn_kv4_cache(2, 2, 64, 16)
    q = _randn((1, 4, 64), 1)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="head dim"):
        attn_fwd_kv4(_randn((1, 4, 128), 1), i, i[:1], i[None], cache, 16)
    with pytest.raises(ValueError, match="pages of 32"):
        attn_fwd_kv4(q, i, i[:1], i[None], cache, 32)
    with pytest.raises(AttnError):  # 3 query heads on 2 kv heads
        attn_fwd_kv4(_randn((1, 3, 64), 1), i, i[:1], i[None], cache, 16)
    with pytest.raises(ValueError, match="requests"):
        attn_fwd_kv4(q, i[:1], i[:1], i[None], cache, 16)
    with pytest.raises(ValueError, match="match"):
        attn_kv4_append(q, q, i, cache, 16)
    with pytest.raises(AttnError):  # no kernel for a cache of this head dim
        attn_fwd_kv4(_randn((1, 4, 320), 1), i, i[:1], i[None], attn_kv4_cache(2, 2, 320, 16), 16)


def test_agrees_with_attn_fwd_on_the_values_read_back():
    # the cached prefix read back for attn_fwd: bfloat16 values of the codes against the codes themselves
    H, Hq, D, P, n = 2, 8, 128, 64, 500
    pages = -(-n // P)
    cache = _random_cache(pages, H, D, P, 12)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    k, v = attn_kv4_read(slots, cache, P)
    q = _randn((n, Hq, D), 13)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    a, la = attn_fwd_kv4(q, dev([0, n]), dev([n]), dev([list(range(pages))]), cache, P)
    b, lb = attn_fwd(q.transpose(0, 1)[None].contiguous(), k[None], v[None], causal=True)
    # K's values move by 2^-8 relative (a score by up to 2^-8 scale sum |q k|, about 0.03 here), V's and both outputs too
    assert (a.float() - b[0].transpose(0, 1).float()).abs().max() <= 0.1
    assert (la - lb[0].T).abs().max() <= 0.1


@pytest.mark.parametrize("lens,nq,H,P,D", [((130,), (1,), 1, 16, 64), ((700, 3, 0, 33), (2, 1, 1, 0), 2, 32, 128), ((1500,), (9,), 1, 64, 192),
                                           ((260,) * 18, (1,) * 18, 8, 16, 64)])
def test_few_short_items(lens, nq, H, P, D):
    # a CTA for each item, merged in shared memory: short tables; the same requests under a wide table take the cut
    # pieces, and both are within the tolerance
    need = max(-(-n // P) for n in lens)
    for width in (need, need + 3000 // P):
        _run(list(lens), list(nq), 4 * H, H, D, P, seed=D, width=width, pad=2)


def test_offsets_past_32_bits():
    # pages that lie more than 2^32 bytes into the cache: written, read and attended over as the first ones are
    H, D, P, n = 8, 128, 16, 150
    page = H * attn_kv4_page_bytes(D, P)
    pages = 2 ** 32 // page + 40
    cache = torch.empty((pages, H, page // H), dtype=torch.uint8, device="cuda")
    small = attn_kv4_cache(10, H, D, P)
    k, v, q = _randn((n, H, D), 1), _randn((n, H, D), 2), _randn((1, 32, D), 3)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    far = [pages - 1 - 3 * i for i in range(10)]
    near = list(range(10))
    outs = []
    for c, ids in ((cache, far), (small, near)):
        slots = dev([ids[t // P] * P + t % P for t in range(n)])
        attn_kv4_append(k, v, slots, c, P)
        outs.append((*attn_kv4_read(slots, c, P), *attn_fwd_kv4(q, dev([0, 1]), dev([n]), dev([ids]), c, P)))
    assert attn_fwd_status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(cache[far, :, :], small[near, :, :])


def test_many_requests():
    # more requests than one warp looks up by itself (128), some without query tokens or without cached tokens
    r = np.random.default_rng(3)
    B = 300
    lens = [int(x) for x in r.integers(0, 90, B)]
    nq = [int(min(x, n)) if n else 0 for x, n in zip(r.integers(0, 3, B), lens)]
    lens[17], nq[17] = 0, 2      # query tokens without a key
    _run(lens, nq, 4, 2, 64, 16, seed=9, pad=3)
    _run(lens, nq, 4, 2, 64, 16, seed=9, width=900)


@pytest.mark.parametrize("H,g,L", [(1, 8, 30000), (2, 1, 9000), (1, 20, 5000)])
def test_long_contexts_cut_into_many_parts(H, g, L):
    _run([L, 40], [1, 2], H * g, H, 128, 32, seed=L, pad=1)


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
def test_many_query_tokens(P, D):
    # more than 64 query rows a request: tiles of 16 rows, one of them ragged, on every page size
    _run([90, 41, 70], [40, 25, 33], 8, 2, D, P, seed=P + D, width=40)
    _run([90, 41, 70], [40, 25, 33], 8, 2, D, P, seed=P + D, causal=False, pad=1)


def test_slots_read_twice_and_tokens_before_the_first_request():
    H, D, P, n = 2, 64, 16, 40
    cache = _random_cache(3, H, D, P, 21)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = attn_kv4_read(dev([7, 7, 30, -1, 7]), cache, P)
    assert torch.equal(k[:, 0], k[:, 1]) and torch.equal(v[:, 0], v[:, 4]) and (k[:, 3] == 0).all()
    q = _randn((6, 4, D), 22)
    out, lse = torch.full_like(q, 9.0), torch.full((6, 4), 9.0, device="cuda")
    attn_fwd_kv4(q, dev([2, 4]), dev([n]), dev([[0, 1, 2]]), cache, P, out=out, lse=lse)
    assert (out[:2] == 9).all() and (out[4:] == 9).all() and (lse[:2] == 9).all() and (lse[4:] == 9).all()
    ref, _ = attn_fwd_kv4(q[2:4], dev([0, 2]), dev([n]), dev([[0, 1, 2]]), cache, P)
    assert torch.equal(out[2:4], ref) and attn_fwd_status() == 0


def test_thousands_of_requests_agree_with_a_few_at_a_time():
    # the lookup of pieces with many requests a thread, against calls of 64 requests (one CTA an item); both are within
    # half precision's 2^-11 of a weight and one bfloat16 rounding, 2^-8 of the values (at most 6)
    r = np.random.default_rng(8)
    B, H, D, P = 5000, 1, 64, 16
    lens = r.integers(0, 70, B)
    pages = 600
    cache = _random_cache(pages, H, D, P, 23)
    table = torch.tensor(r.integers(0, pages, (B, 5)), dtype=torch.int32, device="cuda")
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    q = _randn((B, 2, D), 24)
    out, lse = attn_fwd_kv4(q, cu, lens, table, cache, P)
    assert attn_fwd_status() == 0
    for a in range(0, B, 64 * 7):
        b = min(a + 64, B)
        o, s = attn_fwd_kv4(q[a:b], cu[:b - a + 1], lens[a:b].contiguous(), table[a:b], cache, P)
        assert (out[a:b].float() - o.float()).abs().max() <= 6 * (2.0 ** -8 + 2.0 ** -10)
        seen = torch.isfinite(s)
        assert torch.equal(seen, torch.isfinite(lse[a:b])) and torch.equal(seen[:, 0], lens[a:b] > 0)
        assert (s[seen] - lse[a:b][seen]).abs().max() <= 2.0 ** -16


def test_after_shutdown_and_on_a_stream_handle():
    from exact_attention_attn_gb300 import attn_shutdown
    cache = _random_cache(300, 2, 128, 16, 25)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (_randn((1, 8, 128), 26), dev([0, 1]), dev([4700]), dev([list(range(300))]), cache, 16)
    a, la = attn_fwd_kv4(*args)
    attn_shutdown()
    side = torch.cuda.Stream()
    out, lse = torch.empty_like(a), torch.empty_like(la)
    torch.cuda.synchronize()
    attn_fwd_kv4(*args, out=out, lse=lse, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)
