"""Page calls that are told of the call before: what they refuse, without a GPU."""
import pytest
import torch

from test_abi import Buf, lib  # noqa: F401  (the built library)

ARG = -1


def test_refusals(lib):  # noqa: F811
    p = Buf().p

    def own(after=p, table=p, stride=8, width=8, lens=p, new=p, B=2, P=16, shares=p, pages=9, free=p, cap=4, count=p, co=p, src=p, dst=p, info=p):
        return lib.attn_pages_own_after(after, table, stride, width, lens, new, B, P, shares, pages, free, cap, count, co, src, dst, info, None)

    def assign(after=p, table=p, stride=8, width=8, lens=p, new=p, B=2, P=16, free=p, cap=4, count=p, lo=p, co=p, cu=p, slots=p, pos=p, most=4, info=p):
        return lib.attn_pages_assign_after(after, table, stride, width, lens, new, B, P, free, cap, count, lo, co, cu, slots, pos, most, info, None)

    for after in (p, None):
        for bad in (dict(table=None), dict(stride=7), dict(width=-1), dict(lens=None), dict(new=None), dict(B=-1), dict(B=16385), dict(P=8),
                    dict(free=None), dict(cap=-1), dict(count=None), dict(co=None), dict(info=None)):
            assert own(after, **bad) == ARG and assign(after, **bad) == ARG, bad
        for bad in (dict(shares=None), dict(pages=-1), dict(src=None), dict(dst=None)):
            assert own(after, **bad) == ARG, bad
        for bad in (dict(lo=None), dict(cu=None), dict(slots=None), dict(pos=None), dict(most=-1)):
            assert assign(after, **bad) == ARG, bad


def test_binding_checks_after(lib, monkeypatch):  # noqa: F811
    import exact_attention_attn_gb300 as A
    from exact_attention_attn_gb300 import serving, shared_pages
    calls = []
    for m in (serving, shared_pages):
        monkeypatch.setattr(m, "_cuda", lambda *a, **k: None)
        monkeypatch.setattr(m, "_run", lambda *a: calls.append(a[4]))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    info = i32(2)
    state = (i32(2, 3), i32(2), i32(2))
    own = lambda **k: A.attn_pages_own(*state, i32(4), i32(4), i32(1), 16, **k)  # noqa: E731
    assign = lambda **k: A.attn_pages_assign(*state, i32(4), i32(1), 16, 5, **k)  # noqa: E731
    for call in (own, assign):
        call()
        call(after=info)
        assert calls[-2:] == [None, info.data_ptr()]
        for bad in (i32(1), i32(2, 2), i32(4)[::2]):
            with pytest.raises(ValueError):
                call(after=bad)
    monkeypatch.undo()
    for call in (own, assign):
        with pytest.raises(ValueError, match="CUDA"):
            call(after=info)
    with pytest.raises(TypeError, match="after"):
        serving._after(torch.zeros(2, dtype=torch.int64), -1)
