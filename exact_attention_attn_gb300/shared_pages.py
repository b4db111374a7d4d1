"""Pages that several requests share: ctypes binding of that part of
include/attn.h (argument marshalling only).

A step of a beam search (or of samples that share a prompt) runs

    fork = attn_pages_fork(table, lens, parents, shares, free_pages, free_count, page_size, out=...)
    moved = attn_pages_own(table, lens, new_lens, shares, free_pages, free_count, page_size, out=..., after=fork["info"])
    attn_pages_copy(cache, moved["src"], moved["dst"])
    step = attn_pages_assign(table, lens, new_lens, free_pages, free_count, page_size, max_tokens, after=moved["info"])

and then what serving.py's step runs, without the host knowing a length.
``after`` carries a refusal forward, so that nothing of the step is done: without it
the host has to look at attn_pages_own's info before it appends, since a refused
attn_pages_own leaves pages shared into which attn_pages_assign would put tokens.
``shares`` (int32, one per page of the cache, zeros to begin with) counts the
rows that name a page beyond the first.  Everything else (streams, outputs,
errors) is as in serving.py.
"""
from __future__ import annotations

from .binding import load_library
from .serving import _I32, _U8, _after, _cuda, _dense, _int_outs, _keep, _page_state, _plans, _rows, _run, _sig, _sizes, _written


def _shared_state(table, lens, arg, arg_name, shares, free_pages, free_count, page_size):
    stride, index, B, width, capacity = _page_state(table, lens, arg, arg_name, free_pages, free_count, page_size)
    pages = shares.numel()
    _dense(shares, "shares", _I32, (pages,), index)
    _sizes(pages)
    return stride, index, B, width, capacity, pages


def _planned(name, want, table, lens, arg, arg_name, shares, free_pages, free_count, page_size, out, stream, made_for):
    """The checked sizes of a call and its outputs: looked up where every output is given and the signature is known."""
    key = plan = None
    if out and len(out) == want:
        try:
            key = (name, page_size, _sig(table), _sig(lens), _sig(arg), _sig(shares), _sig(free_pages), _sig(free_count), *out,
                   *map(_sig, out.values()))
            plan = _plans.get(key)
        except AttributeError:  # (an output that is None: made below)
            pass
    if plan:
        return plan, out
    plan = _shared_state(table, lens, arg, arg_name, shares, free_pages, free_count, page_size)
    o = _int_outs(table, made_for(plan), out, stream)
    if key:
        _keep(key, plan)
    return plan, o


def _change_rows(fn, name, table, lens, arg, arg_name, shares, free_pages, free_count, page_size, out, stream):
    plan, o = _planned(name, 3, table, lens, arg, arg_name, shares, free_pages, free_count, page_size, out, stream,
                       lambda p: {"lens": p[2], "free_count": 1, "info": 2})
    stride, index, B, width, capacity, pages = plan
    _run(fn, name, index, stream, table.data_ptr(), stride, width, lens.data_ptr(), arg.data_ptr(), B, page_size,
         shares.data_ptr(), pages, free_pages.data_ptr(), capacity, free_count.data_ptr(), o["lens"].data_ptr(),
         o["free_count"].data_ptr(), o["info"].data_ptr())
    return o


def attn_pages_fork(table, lens, parents, shares, free_pages, free_count, page_size: int, out=None, stream=None) -> dict:
    """Row r becomes a copy of row ``parents[r]`` (its own number: unchanged; -1: emptied), its pages shared.

    ``parents`` int32 [B]; ``shares`` int32 [pages of the cache]; the others as
    attn_pages_assign.  ``table``, ``shares`` and ``free_pages`` are updated in
    place; returns a dict of lens [B], free_count [1] and info [2], of which
    ``out`` may hold any (out["lens"] may be lens)."""
    return _change_rows(load_library().attn_pages_fork, "attn_pages_fork", table, lens, parents, "parents", shares, free_pages,
                        free_count, page_size, out, stream)


def release_shared(table, lens, keep_lens, shares, free_pages, free_count, page_size, out, stream):
    """attn_pages_release with ``shares``: see there."""
    return _change_rows(load_library().attn_pages_release_shared, "attn_pages_release", table, lens, keep_lens, "keep_lens",
                        shares, free_pages, free_count, page_size, out, stream)


def attn_pages_own(table, lens, new_lens, shares, free_pages, free_count, page_size: int, out=None, stream=None,
                   after=None) -> dict:
    """Copy-on-write of the pages that the next attn_pages_assign's tokens go into.

    A request with ``new_lens`` > 0 whose last page is partly filled and shared
    gets a page of its own.  ``table`` and ``shares`` are updated in place; returns
    a dict of free_count [1], src [B], dst [B] (attn_pages_copy's) and info [2].
    ``after`` as attn_pages_assign's: attn_pages_fork's info, if the step has one.
    Refused, it leaves pages shared: give its info to attn_pages_assign."""
    plan, o = _planned("own", 4, table, lens, new_lens, "new_lens", shares, free_pages, free_count, page_size, out, stream,
                       lambda p: {"free_count": 1, "src": p[2], "dst": p[2], "info": 2})
    stride, index, B, width, capacity, pages = plan
    _run(load_library().attn_pages_own_after, "attn_pages_own", index, stream, _after(after, index), table.data_ptr(), stride, width,
         lens.data_ptr(), new_lens.data_ptr(), B, page_size, shares.data_ptr(), pages, free_pages.data_ptr(), capacity,
         free_count.data_ptr(), o["free_count"].data_ptr(), o["src"].data_ptr(), o["dst"].data_ptr(), o["info"].data_ptr())
    return o


def attn_pages_copy(cache, src, dst, stream=None) -> None:
    """Pages ``src`` of a cache copied to pages ``dst`` (int32 [n]; -1: none).

    ``cache`` uint8 [pages, Hkv, page bytes] or, for the caches of several layers
    that share a table, [layers, pages, Hkv, page bytes]; contiguous, of any
    format.  No dst twice, and none that is also a src."""
    key = ("copy", _sig(cache), _sig(src), _sig(dst))
    plan = _plans.get(key)
    if plan is None:
        _cuda(cache, "cache", _U8, 4 if cache.dim() == 4 else 3)
        if not cache.is_contiguous():
            raise ValueError("cache must be contiguous")
        index, (layers, pages, heads, size) = cache.get_device(), cache.shape if cache.dim() == 4 else (1, *cache.shape)
        n = src.numel()
        _dense(src, "src", _I32, (n,), index)
        _dense(dst, "dst", _I32, (n,), index)
        _sizes(pages, layers, n)
        plan = _keep(key, (index, heads * size, pages, layers, pages * heads * size, n))
    index, size, pages, layers, stride, n = plan
    _run(load_library().attn_pages_copy, "attn_pages_copy", index, stream, cache.data_ptr(), size, pages, layers, stride,
         src.data_ptr(), dst.data_ptr(), n)


def attn_pages_compact(table, lens, shares, free_pages, free_count, page_size: int, out=None, stream=None) -> dict:
    """Used pages renumbered to come first: their tables, counts and the moves for attn_pages_copy.

    Updates ``table``, ``shares`` and ``free_pages`` in place unless ``out`` names
    other tensors for them.  Returns a dict of these three, src and dst (the moves,
    -1 behind them; half the number of pages unless given), map [pages] (each
    page's new id, -1 for a free one) and info [2]."""
    given = dict(out) if out else {}
    src = given.get("src")
    moves = shares.numel() // 2 if src is None else src.numel()
    for name, t in (("table", table), ("shares", shares), ("free_pages", free_pages)):
        if given.get(name) is None:
            given[name] = t
    key = plan = None
    if len(given) == 7 and all(t is not None for t in given.values()):
        key = ("compact", page_size, _sig(table), _sig(lens), _sig(shares), _sig(free_pages), _sig(free_count), *given,
               *map(_sig, given.values()))
        plan = _plans.get(key)
    if plan:
        o = given
    else:
        stride, index, B, width, capacity, pages = _shared_state(table, lens, lens, "lens", shares, free_pages, free_count,
                                                                 page_size)
        new = given.pop("table")
        to = _rows(new, index)
        if new.shape != table.shape:
            raise ValueError(f"out's table {tuple(new.shape)} does not match {tuple(table.shape)}")
        _written(new.stride(), new.shape, "out's table")
        _sizes(moves)
        if new.data_ptr() == table.data_ptr() and to != stride:
            raise ValueError("out's table overlaps table")
        o = _int_outs(table, {"shares": pages, "free_pages": capacity, "src": moves, "dst": moves, "map": pages, "info": 2},
                      given, stream)
        o["table"] = new
        plan = stride, to, index, B, width, capacity, pages, moves
        if key:
            _keep(key, plan)
    stride, to, index, B, width, capacity, pages, moves = plan
    _run(load_library().attn_pages_compact, "attn_pages_compact", index, stream, table.data_ptr(), stride, o["table"].data_ptr(),
         to, width, lens.data_ptr(), B, page_size, shares.data_ptr(), o["shares"].data_ptr(), pages, free_pages.data_ptr(),
         o["free_pages"].data_ptr(), capacity, free_count.data_ptr(), o["src"].data_ptr(), o["dst"].data_ptr(), moves,
         o["map"].data_ptr(), o["info"].data_ptr())
    return o
