"""Rotary positions, cache pages, the 4-bit and 8-bit KV caches and attention
over them: ctypes binding of that part of include/attn.h (argument marshalling
only).

A decode or prefill step runs

    step = attn_pages_assign(table, lens, new_lens, free_pages, free_count, page_size, max_tokens)
    q, k = attn_rope(q, k, positions, rope_table)
    attn_kv4_append(k, v, step["slots"], cache, page_size)
    o, lse = attn_fwd_kv4(q, step["cu"], step["lens"], table, cache, page_size)

(or kv8 in the place of kv4) without the host knowing a length.  Every function runs asynchronously on
``stream`` (default: torch's current stream on the tensors' device; a stream or
its handle).  Tensors that a call allocates itself come from that stream's
memory and are kept from reuse until the current stream has passed as well.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .binding import ATTN_OK, AttnError, load_library

_GROUP = 64
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
# A decode step's kernels take a few microseconds, so the calls here are written to cost the host little: each tensor's
# usual form is recognised with a handful of attribute reads, and only another form goes through the checks that say
# what is wrong with it (or that it is fine).
#
# "Plans": what a call passes on besides its pointers (sizes, strides) depends on its tensors' types, shapes, strides
# and devices alone.  It is checked and laid out once for each such signature and looked up afterwards.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_Strides = ctypes.c_longlong * 3
_plans = {}


def _keep(key, plan):
    if len(_plans) >= 4096:
        _plans.clear()
    _plans[key] = plan
    return plan


def _sig(t):
    """All of a tensor that a plan may depend on."""
    return t.dtype, t.get_device(), t.shape, t.stride()


_default_memory = contextlib.nullcontext()


def _memory(stream, index):
    """Where tensors for a call on ``stream`` are allocated: a block of the
    current stream's may still be in use there, ahead of the call."""
    if stream is None:
        return _default_memory
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        handle = 0 if handle == 1 else handle  # two names of the legacy default stream
        stream = torch.cuda.ExternalStream(handle, device=f"cuda:{index}")
    return torch.cuda.stream(stream)


def _keep_for_current(stream, index, *made):
    """The caller uses tensors made for another stream on the current one."""
    if stream is not None:
        for t in made:
            t.record_stream(torch.cuda.current_stream(index))


def _run(fn, what, index, stream, *args):
    """fn(*args, stream) with the tensors' device current."""
    if stream is None and index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            s = torch.cuda.current_stream() if stream is None else stream
            rc = fn(*args, s.cuda_stream if hasattr(s, "cuda_stream") else int(s))
    if rc != ATTN_OK:
        raise AttnError(rc, what)


def _cuda(t, name, dtype, ndim, index=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")


def _dense(t, name, dtype, shape, index):
    """A contiguous tensor of a known shape."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and t.shape == shape:
        return
    _cuda(t, name, dtype, len(shape), index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _sizes(*sizes):
    """The library's sizes are C ints; ctypes would pass the low half of a larger one."""
    if max(sizes) > 0x7fffffff or min(sizes) < -0x80000000:
        raise ValueError(f"sizes {sizes} pass 32 bits")


def _last_dim(t, name):
    """The strides before the last dim, in elements (0 for a dim of size one: it is never stepped along)."""
    s = t.stride()
    if 1 in t.shape:
        if t.shape[-1] > 1 and s[-1] != 1:
            raise ValueError(f"{name}'s last dim must be contiguous")
        return tuple(0 if n == 1 else x for n, x in zip(t.shape[:-1], s[:-1]))
    if s[-1] != 1:
        raise ValueError(f"{name}'s last dim must be contiguous")
    return s[:-1]


def _written(strides, shape, name):
    """A tensor that is written must not hold an element twice (an expanded dim; one without elements holds none)."""
    if 0 in strides and 0 not in shape and any(n > 1 and x == 0 for n, x in zip(shape, strides)):
        raise ValueError(f"{name} is written and must not be expanded")


def _rows(table, index):
    """The row stride of a block table [B, max_pages]."""
    _cuda(table, "table", _I32, 2, index)
    s, n = table.stride(), table.shape
    if n[1] > 1 and s[1] != 1:
        raise ValueError("table's last dim must be contiguous")
    if n[0] > 1:
        return s[0]
    return max(n[1], 1)


# ---------------------------------------------------------------- rotary positions

def attn_rope_axes(sections, interleave: bool = False) -> list:
    """The axis of each frequency: ``sections[a]`` frequencies for axis a, as
    one run after the other, or (``interleave``) the axes in turn while their
    shares last."""
    sections = [int(n) for n in sections]
    if any(n < 0 for n in sections):
        raise ValueError(f"sections {sections} must not be negative")
    if not interleave:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = sections, []
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                out.append(a)
    return out


def attn_rope_table(rot_dim: int, sections=None, base: float = 10000.0, inv_freq=None, interleave: bool = False,
                    device="cuda") -> torch.Tensor:
    """The frequency table of attn_rope, made once per model: int64 [rot_dim / 2, 2].

    ``sections`` (default: one axis) are the frequencies of each axis and sum
    to rot_dim / 2; ``inv_freq`` (floats, rot_dim / 2 of them) overrides
    base^(-2 i / rot_dim)."""
    n = rot_dim // 2
    axis = attn_rope_axes([n] if sections is None else sections, interleave)
    freq = [base ** (-2.0 * i / rot_dim) for i in range(n)] if inv_freq is None else [float(f) for f in inv_freq]
    if rot_dim % 2 or len(axis) != n or len(freq) != n:
        raise ValueError(f"rot_dim {rot_dim} needs {n} frequencies: sections have {len(axis)}, inv_freq {len(freq)}")
    host = torch.empty((n, 2), dtype=torch.int64)
    rc = load_library().attn_rope_table((ctypes.c_double * n)(*freq), (ctypes.c_int * n)(*axis), n,
                                        max(axis, default=0) + 1,
                                        host.data_ptr())
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_table")
    return host.to(device)


def _rope_plan(q, k, positions, table, out_q, out_k):
    index = q.get_device()
    _cuda(q, "q", _BF16, 4)
    B, Hq, N, D = q.shape
    _cuda(positions, "positions", _I32, 3, index)
    axes, b, n = positions.shape
    ps = positions.stride()
    if b != B or n != N:
        raise ValueError(f"positions {tuple(positions.shape)} do not match [axes, {B}, {N}]")
    if N > 1 and ps[2] != 1:
        raise ValueError("positions' last dim must be contiguous")
    half = table.shape[0] if table.dim() else 0
    _dense(table, "table", _I64, (half, 2), index)
    heads, strides = [], []
    for x, out, name in ((q, out_q, "q"), (k, out_k, "k")):
        if x is None:
            heads.append(0)
            strides += [None, None]
            continue
        _cuda(x, name, _BF16, 4, index)
        if x.shape[0] != B or x.shape[2] != N or x.shape[3] != D:
            raise ValueError(f"k {tuple(x.shape)} does not match q {tuple(q.shape)}")
        _cuda(out, "out_" + name, _BF16, 4, index)
        if out.shape != x.shape:
            raise ValueError(f"out_{name} {tuple(out.shape)} does not match {tuple(x.shape)}")
        so = _last_dim(out, "out_" + name)
        _written(so, out.shape, "out_" + name)
        heads.append(x.shape[1])
        strides += [_Strides(*_last_dim(x, name)), _Strides(*so)]
    _sizes(*heads, axes, B, N, D, 2 * half)
    return (index, heads[0], heads[1], *strides, ps[0] if axes > 1 else 0, ps[1] if B > 1 else 0, axes, B, N, D,
            2 * half)


def _rope(q, k, positions, table, adjacent, out_q, out_k, backward, stream, what):
    if out_q is None or (out_k is None and k is not None):
        _cuda(q, "q", _BF16, 4)
        made = []
        with _memory(stream, q.get_device()):
            if out_q is None:
                out_q = torch.empty_like(q)
                made.append(out_q)
            if out_k is None and k is not None:
                out_k = torch.empty_like(k)
                made.append(out_k)
        _keep_for_current(stream, q.get_device(), *made)
    if k is None:
        if out_k is not None:
            raise ValueError("out_k without k")
        key = (_sig(q), None, _sig(positions), _sig(table), _sig(out_q))
    else:
        key = (_sig(q), _sig(k), _sig(positions), _sig(table), _sig(out_q), _sig(out_k))
    plan = _plans.get(key) or _keep(key, _rope_plan(q, k, positions, table, out_q, out_k))
    index, hq, hk, qs, qos, ks, kos, pa, pb, axes, B, N, D, rot = plan
    if k is None:
        kp = kop = None
    else:
        kp, kop = k.data_ptr(), out_k.data_ptr()
    _run(load_library().attn_rope, what, index, stream, q.data_ptr(), qs, out_q.data_ptr(), qos, hq, kp, ks, kop, kos,
         hk, positions.data_ptr(), pa, pb, axes, table.data_ptr(), B, N, D, rot, 1 if adjacent else 0, backward)
    return out_q, out_k


def attn_rope(q, k, positions, table, adjacent: bool = False, out_q=None, out_k=None, stream=None):
    """Rotated q [B, Hq, N, D] and k [B, Hkv, N, D] (or None), bf16, any strides
    with a contiguous last dim (so [T, H, D] as x.transpose(0, 1)[None]).

    ``positions`` int32 [axes, B, N]; ``table`` of attn_rope_table, on the
    same device.  ``out_q``/``out_k`` may be q/k themselves."""
    return _rope(q, k, positions, table, adjacent, out_q, out_k, 0, stream, "attn_rope")


def attn_rope_bwd(dq, dk, positions, table, adjacent: bool = False, out_q=None, out_k=None, stream=None):
    """Gradients of attn_rope's q and k from those of its outputs (the rotation by the opposite angles)."""
    return _rope(dq, dk, positions, table, adjacent, out_q, out_k, 1, stream, "attn_rope_bwd")


# ---------------------------------------------------------------- pages

def _int_outs(like, want, out, stream):
    """The int32 outputs by name (``want``: their lengths): given ones checked, the others made."""
    got, made, index = {}, [], like.get_device()
    if out:
        for name in out:
            if name not in want:
                raise ValueError(f"unknown output {name!r}")
    with _memory(stream, index):
        for name, n in want.items():
            t = out.get(name) if out else None
            if t is None:
                t = torch.empty(n, dtype=_I32, device=like.device)
                made.append(t)
            else:
                _dense(t, name, _I32, (n,), index)
            got[name] = t
    _keep_for_current(stream, index, *made)
    return got


def _page_state(table, lens, arg, arg_name, free_pages, free_count, page_size, max_tokens=0):
    index = table.get_device()
    stride = _rows(table, None)
    B, width = table.shape
    _written(table.stride(), table.shape, "table")
    _dense(lens, "lens", _I32, (B,), index)
    _dense(arg, arg_name, _I32, (B,), index)
    capacity = free_pages.numel()
    _dense(free_pages, "free_pages", _I32, (capacity,), index)
    _dense(free_count, "free_count", _I32, (1,), index)
    _sizes(B, width, capacity, page_size, max_tokens)
    return stride, index, B, width, capacity


def _after(info, index):
    """The pointer of an earlier call's info, or none."""
    if info is None:
        return None
    _dense(info, "after", _I32, (2,), index)
    return info.data_ptr()


def attn_pages_assign(table, lens, new_lens, free_pages, free_count, page_size: int, max_tokens: int, out=None,
                      stream=None, after=None) -> dict:
    """Pages, slots and positions of ``new_lens`` further tokens of each request.

    All int32 on one device: ``table`` [B, max_pages] (updated in place),
    ``lens`` and ``new_lens`` [B], ``free_pages`` [capacity] and ``free_count``
    [1] (a stack of free page ids).  Returns a dict of lens [B], free_count
    [1], cu [B + 1], slots and positions [max_tokens], info [2] (info[0] != 0:
    the step was refused and nothing changed, see ATTN_PAGES_* in
    include/attn.h).  ``out`` may hold any of them; out["lens"] may be lens and
    out["free_count"] free_count, for updates in place.

    ``after``: the info of the step's call before (attn_pages_own's); where that was
    refused, so is this one (out["info"] may be the same tensor)."""
    key = plan = None
    if out and len(out) == 6:
        try:
            key = ("assign", page_size, max_tokens, _sig(table), _sig(lens), _sig(new_lens), _sig(free_pages),
                   _sig(free_count), *out, *map(_sig, out.values()))
            plan = _plans.get(key)
        except AttributeError:  # (an output that is None: made below)
            pass
    if plan:
        o = out
    else:
        plan = _page_state(table, lens, new_lens, "new_lens", free_pages, free_count, page_size, max_tokens)
        o = _int_outs(table, {"lens": plan[2], "free_count": 1, "cu": plan[2] + 1, "slots": max_tokens,
                              "positions": max_tokens, "info": 2}, out, stream)
        if key:
            _keep(key, plan)
    stride, index, B, width, capacity = plan
    _run(load_library().attn_pages_assign_after, "attn_pages_assign", index, stream, _after(after, index), table.data_ptr(),
         stride, width, lens.data_ptr(), new_lens.data_ptr(), B, page_size, free_pages.data_ptr(), capacity,
         free_count.data_ptr(), o["lens"].data_ptr(), o["free_count"].data_ptr(), o["cu"].data_ptr(), o["slots"].data_ptr(),
         o["positions"].data_ptr(), max_tokens, o["info"].data_ptr())
    return o


def attn_pages_release(table, lens, keep_lens, free_pages, free_count, page_size: int, out=None, stream=None,
                       shares=None) -> dict:
    """Requests cut to ``keep_lens`` tokens (0: finished; negative: left alone),
    their pages back on the stack.  ``table`` and ``free_pages`` are updated in
    place; returns a dict of lens [B], free_count [1] and info [2].

    ``shares`` (int32 [pages], updated in place) where requests share pages (attn_pages_fork): a
    page goes back when no other request has it."""
    if shares is not None:
        from .shared_pages import release_shared
        return release_shared(table, lens, keep_lens, shares, free_pages, free_count, page_size, out, stream)
    stride, index, B, width, capacity = _page_state(table, lens, keep_lens, "keep_lens", free_pages, free_count,
                                                        page_size)
    _written(free_pages.stride(), free_pages.shape, "free_pages")
    o = _int_outs(table, {"lens": B, "free_count": 1, "info": 2}, out, stream)
    _run(load_library().attn_pages_release, "attn_pages_release", index, stream, table.data_ptr(), stride, width,
         lens.data_ptr(), keep_lens.data_ptr(), B, page_size, free_pages.data_ptr(), capacity, free_count.data_ptr(),
         o["lens"].data_ptr(), o["free_count"].data_ptr(), o["info"].data_ptr())
    return o


# ---------------------------------------------------------------- the 4-bit and the 8-bit cache
# Their calls take the same arguments; "kv4" and "kv8" name the formats.

def _page_bytes(form, head_dim, page_size):
    what = f"attn_{form}_page_bytes"
    n = int(getattr(load_library(), what)(int(head_dim), int(page_size)))
    if n < 0:
        raise AttnError(n, what)
    return n


def attn_kv4_page_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one kv head of a 4-bit cache."""
    return _page_bytes("kv4", head_dim, page_size)


def attn_kv8_page_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one kv head of an 8-bit cache."""
    return _page_bytes("kv8", head_dim, page_size)


def attn_kv4_cache(num_pages: int, Hkv: int, head_dim: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty 4-bit cache: uint8 [num_pages, Hkv, page bytes]."""
    return torch.zeros((num_pages, Hkv, _page_bytes("kv4", head_dim, page_size)), dtype=torch.uint8, device=device)


def attn_kv8_cache(num_pages: int, Hkv: int, head_dim: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty 8-bit cache: uint8 [num_pages, Hkv, page bytes]."""
    return torch.zeros((num_pages, Hkv, _page_bytes("kv8", head_dim, page_size)), dtype=torch.uint8, device=device)


def _cache(cache, page_size, form):
    """Device, pages, kv heads and head dim of a cache: a page holds 72 bytes per token and group of 64 dims (kv4),
    or two per token and dim and one more a token (kv8)."""
    _cuda(cache, "cache", _U8, 3)
    if not cache.is_contiguous():
        raise ValueError("cache must be contiguous")
    pages, heads, size = cache.shape
    if page_size >= 1:
        n, rest = divmod(size, page_size)
        groups, odd = divmod(n, 72) if form == "kv4" else divmod(n - 1, 2 * _GROUP)
    if page_size < 1 or rest or odd or groups < 1:
        raise ValueError(f"cache {tuple(cache.shape)} is not one of pages of {page_size} tokens")
    return cache.get_device(), pages, heads, groups * _GROUP


def _view(t, name, shape, index):
    """The strides of a bf16 [.., .., D] view of a known shape."""
    if not (t.dtype is _BF16 and t.shape == shape and t.get_device() == index):
        _cuda(t, name, _BF16, 3, index)
        raise ValueError(f"{name} {tuple(t.shape)} does not match {tuple(shape)}")
    return _last_dim(t, name)


def _append(fn, what, form, k, v, slots, cache, page_size, stream):
    key = (what, page_size, _sig(k), _sig(v), _sig(slots), _sig(cache))
    plan = _plans.get(key)
    if plan is None:
        index, pages, H, D = _cache(cache, page_size, form)
        T = slots.numel()
        _dense(slots, "slots", _I32, (T,), index)
        ks, vs = _view(k, "k", (T, H, D), index), _view(v, "v", (T, H, D), index)
        _sizes(pages, T, H, D)
        plan = _keep(key, (index, *ks, *vs, pages, T, H, D))
    index, kt, kh, vt, vh, pages, T, H, D = plan
    _run(fn, what, index, stream, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(), cache.data_ptr(), pages, T, H, D,
         page_size)


def attn_kv4_append(k, v, slots, cache, page_size: int, stream=None) -> None:
    """Quantises k and v (bf16 [T, Hkv, D], any strides with a contiguous last
    dim) into the cache's slots (int32 [T]; -1 skips a token; no slot twice)."""
    _append(load_library().attn_kv4_append, "attn_kv4_append", "kv4", k, v, slots, cache, page_size, stream)


def attn_kv8_append(k, v, slots, cache, page_size: int, stream=None) -> None:
    """Quantises k and v (bf16 [T, Hkv, D], any strides with a contiguous last
    dim) into an 8-bit cache's slots (int32 [T]; -1 skips a token; no slot twice;
    the tokens of a block of 16 slots within 16 consecutive ones, as
    attn_pages_assign lists them).

    A block's scale is that of its largest value; where a token needs a larger one,
    the codes held are rounded again.  Writing a block's first slot clears the block."""
    _append(load_library().attn_kv8_append, "attn_kv8_append", "kv8", k, v, slots, cache, page_size, stream)


def _read(fn, what, form, slots, cache, page_size, out_k, out_v, stream):
    if out_k is None or out_v is None:
        index, _, H, D = _cache(cache, page_size, form)
        made = []
        with _memory(stream, index):
            if out_k is None:
                out_k = torch.empty((H, slots.numel(), D), dtype=_BF16, device=cache.device)
                made.append(out_k)
            if out_v is None:
                out_v = torch.empty((H, slots.numel(), D), dtype=_BF16, device=cache.device)
                made.append(out_v)
        _keep_for_current(stream, index, *made)
    key = (what, page_size, _sig(slots), _sig(cache), _sig(out_k), _sig(out_v))
    plan = _plans.get(key)
    if plan is None:
        index, pages, H, D = _cache(cache, page_size, form)
        T = slots.numel()
        _dense(slots, "slots", _I32, (T,), index)
        ks, vs = _view(out_k, "out_k", (H, T, D), index), _view(out_v, "out_v", (H, T, D), index)
        _written(ks, out_k.shape, "out_k")
        _written(vs, out_v.shape, "out_v")
        _sizes(pages, T, H, D)
        plan = _keep(key, (index, *ks, *vs, pages, T, H, D))
    index, kh, kt, vh, vt, pages, T, H, D = plan
    _run(fn, what, index, stream, cache.data_ptr(), pages, slots.data_ptr(), out_k.data_ptr(), kh, kt, out_v.data_ptr(), vh, vt, T,
         H, D, page_size)
    return out_k, out_v


def attn_kv4_read(slots, cache, page_size: int, out_k=None, out_v=None, stream=None):
    """K and V of the slots (int32 [T]) as bf16 [Hkv, T, D]: k[None], v[None]
    are attn_fwd's operands for a cached prefix.  Slot -1 reads as zeros."""
    return _read(load_library().attn_kv4_read, "attn_kv4_read", "kv4", slots, cache, page_size, out_k, out_v, stream)


def attn_kv8_read(slots, cache, page_size: int, out_k=None, out_v=None, stream=None):
    """K and V of an 8-bit cache's slots: as attn_kv4_read."""
    return _read(load_library().attn_kv8_read, "attn_kv8_read", "kv8", slots, cache, page_size, out_k, out_v, stream)


def _attend(fn, what, form, q, cu, lens, table, cache, page_size, scale, causal, out, lse, stream):
    if out is None or lse is None:
        index = cache.get_device()
        if stream is not None:
            _cuda(q, "q", _BF16, 3, index)
        made = []
        with _memory(stream, index):
            if out is None:
                out = torch.empty(q.shape, dtype=_BF16, device=q.device)
                made.append(out)
            if lse is None:
                lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
                made.append(lse)
        _keep_for_current(stream, index, *made)
    key = (what, page_size, _sig(q), _sig(cu), _sig(lens), _sig(table), _sig(cache), _sig(out), _sig(lse))
    plan = _plans.get(key)
    if plan is None:
        index, pages, H, D = _cache(cache, page_size, form)
        _cuda(q, "q", _BF16, 3, index)
        T, Hq = q.shape[:2]
        if q.shape[2] != D:
            raise ValueError(f"q {tuple(q.shape)} does not match the cache's head dim {D}")
        qs = _view(q, "q", (T, Hq, D), index)
        stride = _rows(table, index)
        B, width = table.shape
        if cu.shape != (B + 1,) or lens.shape != (B,):
            raise ValueError(f"cu {tuple(cu.shape)} / lens {tuple(lens.shape)} do not match {B} requests "
                             "(rows of table)")
        _dense(cu, "cu", _I32, (B + 1,), index)
        _dense(lens, "lens", _I32, (B,), index)
        _dense(out, "out", _BF16, (T, Hq, D), index)
        _dense(lse, "lse", _F32, (T, Hq), index)
        _sizes(width, pages, B, T, Hq, H, D)
        plan = _keep(key, (index, *qs, stride, width, pages, B, T, Hq, H, D, 1.0 / math.sqrt(D)))
    index, qt, qh, stride, width, pages, B, T, Hq, H, D, usual = plan
    _run(fn, what, index, stream, q.data_ptr(), qt, qh, cu.data_ptr(), lens.data_ptr(), table.data_ptr(), stride, width,
         cache.data_ptr(), pages, out.data_ptr(), lse.data_ptr(), B, T, Hq, H, D, page_size, usual if scale is None else scale,
         1 if causal else 0)
    return out, lse


def attn_fwd_kv4(q, cu, lens, table, cache, page_size: int, scale: float | None = None, causal: bool = True, out=None,
                 lse=None, stream=None):
    """O [T, Hq, D] (bf16), LSE [T, Hq] (fp32): attention of q (bf16 [T, Hq, D])
    over the cached tokens of each request.

    ``cu`` [B + 1], ``lens`` [B] and ``table`` [B, max_pages] int32 as
    attn_pages_assign gives them: request r has query tokens cu[r] .. cu[r+1] - 1
    and lens[r] cached tokens, theirs among them (``causal``: bottom-right
    aligned, as attn_fwd).  Rows outside cu[0] .. cu[B] are left as they were.
    Head dims 64, 128, 192, 256."""
    return _attend(load_library().attn_fwd_kv4, "attn_fwd_kv4", "kv4", q, cu, lens, table, cache, page_size, scale, causal, out,
                   lse, stream)


def attn_fwd_kv8(q, cu, lens, table, cache, page_size: int, scale: float | None = None, causal: bool = True, out=None,
                 lse=None, stream=None):
    """O, LSE of q over an 8-bit cache: as attn_fwd_kv4."""
    return _attend(load_library().attn_fwd_kv8, "attn_fwd_kv8", "kv8", q, cu, lens, table, cache, page_size, scale, causal, out,
                   lse, stream)
