"""Refusals of the rotary, page, cache and kv4 entry points, without a GPU:
through the C ABI, and through the binding's own checks."""
import ctypes as C

import pytest
import torch

from test_abi import Buf, lib  # noqa: F401  (the built library)

ARG, ALIGN = -1, -2


def strides(*s):
    return (C.c_longlong * 3)(*s)


def test_rope_table(lib):  # noqa: F811
    n = 3
    out = (C.c_longlong * 6)()
    freq, axis = (C.c_double * n)(1.0, 0.5, 7.0), (C.c_int * n)(0, 1, 1)
    assert lib.attn_rope_table(freq, axis, n, 2, out) == 0
    turns = [(v % (1 << 64)) / 2.0 ** 64 for v in out[0::2]]
    two_pi = 6.283185307179586
    for got, f in zip(turns, (1.0, 0.5, 7.0)):
        assert abs(got - (f / two_pi) % 1.0) < 1e-15
    assert list(out[1::2]) == [0, 1, 1]
    assert lib.attn_rope_table((C.c_double * 1)(-1e-30), axis, 1, 2, out) == 0 and out[0] == 0  # a whole turn is none
    assert lib.attn_rope_table(freq, axis, n, 1, out) == ARG          # an axis past the last
    assert lib.attn_rope_table((C.c_double * n)(1, float("inf"), 1), axis, n, 2, out) == ARG
    assert lib.attn_rope_table(freq, axis, 513, 2, out) == ARG
    assert lib.attn_rope_table(freq, axis, n, 9, out) == ARG
    assert lib.attn_rope_table(None, axis, n, 2, out) == ARG
    assert lib.attn_rope_table(None, None, 0, 1, None) == 0


def test_rope_refusals(lib):  # noqa: F811
    p = Buf().p
    s = strides(512, 64, 256)

    def rope(q=p, qs=s, o=p, os=s, Hq=4, k=None, Hkv=0, pos=p, pa=8, pb=0, axes=1, table=p, B=1, N=2, D=64, rot=64,
             adj=0, bwd=0):
        return lib.attn_rope(q, qs, o, os, Hq, k, s, k, s, Hkv, pos, pa, pb, axes, table, B, N, D, rot, adj, bwd, None)

    for bad in (dict(D=96), dict(D=1088), dict(rot=8), dict(rot=24), dict(rot=80), dict(axes=0), dict(axes=9), dict(adj=2),
                dict(bwd=-1), dict(B=-1), dict(N=-1), dict(Hq=-1), dict(pa=-1), dict(pb=-4), dict(q=None), dict(o=None),
                dict(qs=None), dict(Hkv=2), dict(pos=None), dict(table=None), dict(qs=strides(512, -64, 256)),
                dict(os=strides(512, 64, 264))):  # in place with another layout
        assert rope(**bad) == ARG, bad
    for bad in (dict(q=p + 2), dict(o=p + 8), dict(qs=strides(512, 68, 256)), dict(os=strides(4, 64, 256)),
                dict(table=p + 8), dict(pos=p + 2)):
        assert rope(**bad) == ALIGN, bad
    assert rope(B=0, q=None) == 0 and rope(N=0, q=None) == 0 and rope(Hq=0, q=None) == 0


def test_sizes_near_32_bits_are_refused(lib):  # noqa: F811
    # a CTA's last tokens would have numbers past 2^31 - 1, and products of sizes pass 64 bits
    p = Buf().p
    s = strides(0, 0, 0)
    most = 2 ** 31 - 1

    def rope(B, N, Hq, Hk):
        return lib.attn_rope(p, s, p, s, Hq, p, s, p, s, Hk, p, 0, 0, 1, p, B, N, 64, 64, 0, 0, None)

    assert rope(1, most, 1, 0) == ARG and rope(1, most - 2, 1, 0) == ARG
    assert rope(1 << 16, 1 << 17, most, 1) == ARG      # 2^64 + 2^33 rows
    assert rope(most, most, most, most) == ARG
    for T in (most, most - 30):
        assert lib.attn_kv4_append(p, 0, 0, p, 0, 0, p, p, 4, T, 1, 64, 16, None) == ARG
        assert lib.attn_kv4_read(p, 4, p, p, 0, 0, p, 0, 0, T, 1, 64, 16, None) == ARG


def test_pages_refusals(lib):  # noqa: F811
    p = Buf().p

    def assign(table=p, stride=8, width=8, lens=p, new=p, B=2, P=16, free=p, cap=4, count=p, lo=p, co=p, cu=p, slots=p,
               pos=p, most=4, info=p):
        return lib.attn_pages_assign(table, stride, width, lens, new, B, P, free, cap, count, lo, co, cu, slots, pos,
                                     most, info, None)

    def release(table=p, stride=8, width=8, lens=p, keep=p, B=2, P=16, free=p, cap=4, count=p, lo=p, co=p, info=p):
        return lib.attn_pages_release(table, stride, width, lens, keep, B, P, free, cap, count, lo, co, info, None)

    both = [dict(table=None), dict(stride=7), dict(width=-1), dict(width=1 << 28, stride=1 << 28), dict(lens=None),
            dict(B=-1), dict(B=16385), dict(P=8), dict(P=48), dict(P=128), dict(free=None), dict(cap=-1),
            dict(count=None), dict(lo=None), dict(co=None), dict(info=None)]
    for bad in both + [dict(new=None), dict(cu=None), dict(slots=None), dict(pos=None), dict(most=-1)]:
        assert assign(**bad) == ARG, bad
    for bad in both + [dict(keep=None)]:
        assert release(**bad) == ARG, bad


def test_kv4_refusals(lib):  # noqa: F811
    p = Buf().p
    assert lib.attn_kv4_page_bytes(128, 16) == 2304 and lib.attn_kv4_page_bytes(1024, 64) == 73728
    for d, s in ((96, 16), (0, 16), (1088, 16), (64, 8), (64, 48), (64, 0)):
        assert lib.attn_kv4_page_bytes(d, s) == ARG

    def append(k=p, kt=64, kh=64, v=p, vt=64, vh=64, slots=p, cache=p, pages=4, T=1, H=1, D=64, P=16):
        return lib.attn_kv4_append(k, kt, kh, v, vt, vh, slots, cache, pages, T, H, D, P, None)

    def read(cache=p, pages=4, slots=p, k=p, kh=64, kt=64, v=p, vh=64, vt=64, T=1, H=1, D=64, P=16):
        return lib.attn_kv4_read(cache, pages, slots, k, kh, kt, v, vh, vt, T, H, D, P, None)

    for call in (append, read):
        for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(pages=-1), dict(T=-1),
                    dict(H=0), dict(H=65536), dict(D=96), dict(P=24), dict(kt=-8), dict(vh=-8), dict(pages=1 << 27)):
            assert call(**bad) == ARG, (call, bad)
        for bad in (dict(k=p + 2), dict(v=p + 8), dict(cache=p + 4), dict(slots=p + 1), dict(kh=4), dict(vt=12)):
            assert call(**bad) == ALIGN, (call, bad)
        assert call(T=0, k=None, v=None, slots=None) == 0

    def fwd(q=p, qt=256, qh=64, cu=p, lens=p, table=p, stride=4, width=4, cache=p, pages=4, o=p, lse=p, B=1, T=1, Hq=4,
            H=2, D=64, P=16, scale=0.125, causal=1):
        return lib.attn_fwd_kv4(q, qt, qh, cu, lens, table, stride, width, cache, pages, o, lse, B, T, Hq, H, D, P,
                                scale, causal, None)

    for bad in (dict(q=None), dict(o=None), dict(lse=None), dict(cu=None), dict(lens=None), dict(table=None),
                dict(cache=None), dict(stride=3), dict(width=-1), dict(pages=-1), dict(B=-1), dict(B=16385), dict(T=-1),
                dict(Hq=0), dict(H=0), dict(Hq=5), dict(D=96), dict(D=320), dict(D=0), dict(P=8), dict(causal=2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(qt=-8), dict(T=1 << 30, Hq=8, H=1)):
        assert fwd(**bad) == ARG, bad
    for bad in (dict(q=p + 2), dict(o=p + 8), dict(lse=p + 4), dict(cache=p + 8), dict(qh=4), dict(qt=12), dict(cu=p + 2),
                dict(lens=p + 1), dict(table=p + 2)):
        assert fwd(**bad) == ALIGN, bad
    assert fwd(B=0, q=None) == 0 and fwd(T=0, q=None) == 0


def test_binding_refuses_sizes_past_32_bits(lib, monkeypatch):  # noqa: F811
    # a size that 32 bits do not hold must not reach the library as its low half (meta tensors: no memory behind them)
    import exact_attention_attn_gb300 as A
    from exact_attention_attn_gb300 import serving
    monkeypatch.setattr(serving, "_cuda", lambda *a: None)
    monkeypatch.setattr(serving, "_dense", lambda *a: None)
    monkeypatch.setattr(serving, "_run", lambda *a: pytest.fail("called"))
    bf, i32, big = torch.bfloat16, torch.int32, 2 ** 32 + 1
    one, many = torch.zeros(1, dtype=i32), torch.empty(big, dtype=i32, device="meta")
    cache, table = A.attn_kv4_cache(2, 1, 64, 16, device="cpu"), A.attn_rope_table(64, device="cpu")
    x = torch.empty((big, 1, 64), dtype=bf, device="meta")
    y = x.transpose(0, 1)
    with pytest.raises(ValueError, match="32 bits"):
        A.attn_kv4_append(x, x, many, cache, 16)
    with pytest.raises(ValueError, match="32 bits"):
        A.attn_kv4_read(many, cache, 16, out_k=y, out_v=y)
    with pytest.raises(ValueError, match="32 bits"):
        A.attn_fwd_kv4(x, one.expand(2), one, one[None], cache, 16, out=x, lse=one)
    with pytest.raises(ValueError, match="32 bits"):
        A.attn_rope(y[None], None, many[None, None], table, out_q=y[None])
    for call in (lambda: A.attn_pages_assign(one[None], one, one, many, one, 16, 4),
                 lambda: A.attn_pages_assign(one[None], one, one, one, one, 2 ** 32 + 16, 4),
                 lambda: A.attn_pages_assign(one[None], one, one, one, one, 16, big),
                 lambda: A.attn_pages_assign(many[None], one, one, one, one, 16, 4),
                 lambda: A.attn_pages_release(one[None], one, one, many, one, 16),
                 lambda: A.attn_pages_release(one[None], one, one, one, one, 2 ** 32 + 16)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_binding_refuses_other_ranks(lib):  # noqa: F811
    import exact_attention_attn_gb300 as A
    cache, one = A.attn_kv4_cache(2, 1, 64, 16, device="cpu"), torch.zeros(1, dtype=torch.int32)
    x, scalar = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros((), dtype=torch.int32)
    for call in (lambda: A.attn_kv4_append(x, x, scalar, cache, 16), lambda: A.attn_kv4_read(scalar, cache, 16),
                 lambda: A.attn_fwd_kv4(x[0, 0], one, one, one[None], cache, 16),
                 lambda: A.attn_fwd_kv4(x[0], one, one, one[None], cache, 16),
                 lambda: A.attn_fwd_kv4(x, scalar, one, one, cache, 16),
                 lambda: A.attn_pages_assign(one[None], one, one, scalar, one, 16, 4),
                 lambda: A.attn_pages_release(one, one, one, one, one, 16),
                 lambda: A.attn_rope(x[None], None, one[None, None], scalar)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_cpu_tensors_and_shapes(lib):  # noqa: F811
    import exact_attention_attn_gb300 as A
    bf, i32 = torch.bfloat16, torch.int32
    q, pos = torch.zeros(1, 2, 3, 64, dtype=bf), torch.zeros(1, 1, 3, dtype=i32)
    table = A.attn_rope_table(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rope(q, None, pos, table)
    with pytest.raises(TypeError, match="bfloat16"):
        A.attn_rope(q.half(), None, pos, table)
    with pytest.raises(ValueError, match="frequencies"):
        A.attn_rope_table(64, [8, 8], device="cpu")
    with pytest.raises(A.AttnError):
        A.attn_rope_table(64, inv_freq=[float("nan")] * 32, device="cpu")
    assert A.attn_rope_axes([3, 1, 2]) == [0, 0, 0, 1, 2, 2]
    assert A.attn_rope_axes([3, 1, 2], interleave=True) == [0, 1, 2, 0, 2, 0]
    with pytest.raises(A.AttnError):
        A.attn_kv4_page_bytes(96, 16)
    cache = A.attn_kv4_cache(2, 1, 64, 16, device="cpu")
    assert cache.shape == (2, 1, 1152)
    one = torch.zeros(1, dtype=i32)
    for call in (lambda: A.attn_kv4_append(q[0], q[0], one, cache, 16), lambda: A.attn_kv4_read(one, cache, 16),
                 lambda: A.attn_fwd_kv4(q[0], one, one, one[None], cache, 16),
                 lambda: A.attn_pages_assign(one[None], one, one, one, one, 16, 4),
                 lambda: A.attn_pages_release(one[None], one, one, one, one, 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_outputs_given_as_none_are_made(monkeypatch):
    # six entries, some of them None, as with fewer
    import exact_attention_attn_gb300 as A
    from exact_attention_attn_gb300 import serving
    monkeypatch.setattr(serving, "_cuda", lambda *a, **k: None)
    calls = []
    monkeypatch.setattr(serving, "_run", lambda *a: calls.append(a))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    names = ("lens", "free_count", "cu", "slots", "positions", "info")
    for given in ({}, {n: None for n in names}, {**{n: None for n in names}, "slots": i32(5)}):
        o = A.attn_pages_assign(i32(2, 3), i32(2), i32(2), i32(4), i32(1), 16, 5, out=given)
        assert {n: tuple(o[n].shape) for n in names} == {"lens": (2,), "free_count": (1,), "cu": (3,), "slots": (5,),
                                                         "positions": (5,), "info": (2,)}
        assert given.get("slots") is None or o["slots"] is given["slots"]
    assert len(calls) == 3


def test_a_table_without_columns_is_no_expanded_one(monkeypatch):
    # a tensor without elements may have any strides (those made from an empty array are 0)
    import numpy as np

    import exact_attention_attn_gb300 as A
    from exact_attention_attn_gb300 import serving
    monkeypatch.setattr(serving, "_cuda", lambda *a, **k: None)
    calls = []
    monkeypatch.setattr(serving, "_run", lambda *a: calls.append(a))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    table = torch.tensor(np.zeros((5, 0)), dtype=torch.int32)
    assert table.stride(0) == 0
    A.attn_pages_assign(table, i32(5), i32(5), i32(4), i32(1), 16, 0)
    A.attn_pages_release(table, i32(5), i32(5), i32(4), i32(1), 16)
    with pytest.raises(ValueError, match="expanded"):
        A.attn_pages_assign(i32(1, 3).expand(5, 3), i32(5), i32(5), i32(4), i32(1), 16, 0)
    assert len(calls) == 2
