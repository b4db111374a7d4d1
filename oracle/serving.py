"""Oracle for rotary positions, cache pages, the 4-bit cache and attention over
it (test infrastructure only; numpy float64 and plain loops).

Only ``tests/`` may import this module.  It shares no code with the CUDA path.

Readings: the definitions in include/attn.h.  A bfloat16 value is rounded to
nearest, ties to even, from float64.
"""
from __future__ import annotations

import numpy as np

from .attention import attention

GROUP = 64


def to_bf16(x):
    """Nearest bfloat16 of each float64 (ties to even; finite inputs in range)."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)                       # x = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.round(x / step) * step         # np.round: ties to even


def bf16_of_bits(b):
    return (np.asarray(b, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


# ---------------------------------------------------------------- rotary positions

def rope(x, positions, inv_freq, axis, adjacent=False, backward=False):
    """x [B, H, N, D], positions [A, B, N], inv_freq and axis [rot / 2]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        phi = np.asarray(positions[axis[i]], dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        if backward:
            s = -s
        u, w = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[..., u] = x[..., u] * c - x[..., w] * s
        y[..., w] = x[..., w] * c + x[..., u] * s
    return y


# ---------------------------------------------------------------- pages

def pages_assign(table, lens, new, free, count, P, max_tokens):
    """The step's outputs and the new table, or the refusal bits: a dict."""
    B, width = table.shape
    bits = 0
    if not 0 <= count <= len(free):
        bits |= 8
    good = [0 <= lens[r] and 0 <= new[r] and int(lens[r]) + int(new[r]) <= width * P for r in range(B)]
    if not all(good):
        bits |= 1
    need = [-(-(int(lens[r]) + int(new[r])) // P) - -(-int(lens[r]) // P) if good[r] else 0 for r in range(B)]
    total = sum(int(new[r]) for r in range(B) if good[r])
    if total > max_tokens:
        bits |= 2
    if sum(need) > count:
        bits |= 4
    slots, positions = np.full(max_tokens, -1), np.zeros(max_tokens, dtype=np.int64)
    if bits:
        return {"info": [bits, 0], "table": table.copy(), "lens": np.array(lens), "free_count": count,
                "cu": np.zeros(B + 1, dtype=np.int64), "slots": slots, "positions": positions}
    table, at, n, cu = table.copy(), count, 0, [0]
    for r in range(B):
        for j in range(need[r]):
            at -= 1
            table[r, -(-int(lens[r]) // P) + j] = free[at]
        for p in range(int(lens[r]), int(lens[r]) + int(new[r])):
            page = int(table[r, p // P])
            slots[n], positions[n] = page * P + p % P if 0 <= page < 2 ** 31 // P else -2, p
            n += 1
        cu.append(n)
    return {"info": [0, n], "table": table, "lens": np.array(lens) + np.array(new), "free_count": at,
            "cu": np.array(cu), "slots": slots, "positions": positions}


def pages_release(table, lens, keep, free, count, P):
    B, width = table.shape
    bits = 0 if 0 <= count <= len(free) else 8
    good = [0 <= lens[r] <= width * P for r in range(B)]
    if not all(good):
        bits |= 1
    cut = [good[r] and 0 <= keep[r] < lens[r] for r in range(B)]
    give = [(r, j) for r in range(B) if cut[r] for j in range(-(-int(keep[r]) // P), -(-int(lens[r]) // P))]
    if count + len(give) > len(free):
        bits |= 4
    if bits:
        return {"info": [bits, 0], "table": table.copy(), "lens": np.array(lens), "free_count": count, "free": free.copy()}
    table, free = table.copy(), free.copy()
    for r, j in give:
        free[count] = table[r, j]
        table[r, j] = -1
        count += 1
    return {"info": [0, len(give)], "table": table, "lens": np.where(cut, keep, lens), "free_count": count, "free": free}


# ---------------------------------------------------------------- the 4-bit cache

def kv4_scale(m, hi):
    """The scale of groups with minima m and maxima hi: the bfloat16 number nearest
    to (hi - m) / 15, from float64.  Where that lies so close to the middle of two
    numbers that float32 cannot tell (2^-22 relative), the format's own rule
    decides: the float32 product of (hi - m) / 16, each step rounded, with the
    float32 number nearest to 16 / 15, then rounded with ties to even."""
    m, hi = np.asarray(m, dtype=np.float64), np.asarray(hi, dtype=np.float64)
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        exact = (hi - m) / 15
        low, high = to_bf16(exact * (1 - 2.0 ** -22)), to_bf16(exact * (1 + 2.0 ** -22))
        rule = ((hi / 16).astype(f) - (m / 16).astype(f)) * f(1 / 0.9375)
        return np.where(low == high, to_bf16(exact), np.clip(to_bf16(rule.astype(np.float64)), low, high))


def kv4_quantise(x):
    """x [..., D]: codes [..., D], scale and minimum [..., D / 64], and the exact
    quotients (x - m) / s that the codes round (0 where s = 0)."""
    x = np.asarray(x, dtype=np.float64)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    m, hi = y.min(-1), y.max(-1)
    s = kv4_scale(m, hi)
    q = np.where(s[..., None] > 0, (y - m[..., None]) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    codes = np.clip(np.round(q), 0, 15).astype(np.int64)
    return codes.reshape(x.shape), s, m, q.reshape(x.shape)


def kv4_unpack(cache, D, P):
    """cache uint8 [pages, H, bytes]: K's (codes [pages, H, P, D], scales, minima
    [pages, H, P, D / 64]), then V's."""
    G = D // GROUP
    n, H, size = cache.shape
    if size != 72 * G * P:
        raise ValueError("not a cache of this head dim and page size")
    out = []
    for at in (0, 36 * G * P):
        byte = cache[:, :, at:at + 32 * G * P].reshape(n, H, G, P, 32).astype(np.int64)
        codes = np.empty((n, H, G, P, GROUP), dtype=np.int64)
        codes[..., 0::2], codes[..., 1::2] = byte % 16, byte // 16
        pair = np.ascontiguousarray(cache[:, :, at + 32 * G * P:at + 36 * G * P]).view(np.uint16).reshape(n, H, G, P, 2)
        pair = bf16_of_bits(pair)
        out.append((codes.transpose(0, 1, 3, 2, 4).reshape(n, H, P, D), pair[..., 0].transpose(0, 1, 3, 2),
                    pair[..., 1].transpose(0, 1, 3, 2)))
    return out


def kv4_values(codes, s, m):
    c = codes.reshape(codes.shape[:-1] + (codes.shape[-1] // GROUP, GROUP)).astype(np.float64)
    return (c * s[..., None] + m[..., None]).reshape(codes.shape)


def attention_requests(q, cu, lens, table, k, v, P, scale, causal):
    """q [T, Hq, D], k and v [pages, Hkv, P, D] (values).  Returns O [T, Hq, D]
    and LSE [T, Hq]; NaN in the rows of tokens that no request has."""
    q = np.asarray(q, dtype=np.float64)
    O, L = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for r in range(len(lens)):
        a, b, n = int(cu[r]), int(cu[r + 1]), int(lens[r])
        if b == a:
            continue
        ids = [int(i) for i in table[r][:-(-n // P)]]
        kr = k[ids].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :n]
        vr = v[ids].transpose(1, 0, 2, 3).reshape(v.shape[1], -1, v.shape[3])[:, :n]
        o, lse = attention(q[a:b].transpose(1, 0, 2)[None], kr[None], vr[None], scale, causal)
        O[a:b], L[a:b] = o[0].transpose(1, 0, 2), lse[0].T
    return O, L
