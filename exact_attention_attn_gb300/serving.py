"""Rotary positions, cache pages, the 4-bit KV cache and attention over it:
ctypes binding of that part of include/attn.h (argument marshalling only).

A decode or prefill step runs

    step = attn_pages_assign(table, lens, new_lens, free_pages, free_count, page_size, max_tokens)
    q, k = attn_rope(q, k, positions, rope_table)
    attn_kv4_append(k, v, step["slots"], cache, page_size)
    o, lse = attn_fwd_kv4(q, step["cu"], step["lens"], table, cache, page_size)

without the host knowing a length.  Every function runs asynchronously on
``stream`` (default: torch's current stream on the tensors' device); tensors
that it allocates itself are kept from reuse until that stream has passed.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import ATTN_OK, AttnError, load_library

_GROUP = 64
_Strides = ctypes.c_longlong * 3


class _On:
    """The tensors' device made current, and the stream's handle."""
    __slots__ = ("device", "stream", "guard", "handle")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        s = torch.cuda.current_stream() if self.stream is None else self.stream
        self.handle = s.cuda_stream if hasattr(s, "cuda_stream") else int(s)
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False

    def keep(self, *tensors):
        """Allocated here for the current stream, used on another one."""
        if self.stream is not None and isinstance(self.stream, torch.cuda.Stream):
            for t in tensors:
                t.record_stream(self.stream)


def _cuda(t, name, dtype, ndim, device=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _dense(t, name, dtype, ndim, device=None):
    _cuda(t, name, dtype, ndim, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims_last(t, name):
    """The strides before the last dim, in elements; a dim of size one has none that matters."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dim must be contiguous")
    return [0 if n == 1 else s for n, s in zip(t.shape[:-1], t.stride()[:-1])]


def _written(t, name):
    """A tensor that is written must not hold an element twice (an expanded dim)."""
    if any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name} is written and must not be expanded")


def _done(rc, what):
    if rc != ATTN_OK:
        raise AttnError(rc, what)


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
    axes = max(axis, default=0) + 1
    _done(load_library().attn_rope_table((ctypes.c_double * n)(*freq), (ctypes.c_int * n)(*axis), n, axes,
                                         host.data_ptr()), "attn_rope_table")
    return host.to(device)


def _rope(q, k, positions, table, adjacent, out_q, out_k, backward, stream, what):
    lib = load_library()
    dev = q.device
    _cuda(q, "q", torch.bfloat16, 4)
    B, Hq, N, D = q.shape
    _cuda(positions, "positions", torch.int32, 3, dev)
    if positions.shape[1] != B or positions.shape[2] != N:
        raise ValueError(f"positions {tuple(positions.shape)} do not match [axes, {B}, {N}]")
    ps = positions.stride()
    if N > 1 and ps[2] != 1:
        raise ValueError("positions' last dim must be contiguous")
    _dense(table, "table", torch.int64, 2, dev)
    if table.shape[1] != 2:
        raise ValueError(f"table must be [rot_dim / 2, 2], got {tuple(table.shape)}")
    pairs, made = [], []
    for x, out, name in ((q, out_q, "q"), (k, out_k, "k")):
        if x is None:
            if out is not None:
                raise ValueError(f"out_{name} without {name}")
            pairs.append((None, None, None, None, 0, None))
            continue
        if x is not q:
            _cuda(x, name, torch.bfloat16, 4, dev)
            if x.shape[0] != B or x.shape[2] != N or x.shape[3] != D:
                raise ValueError(f"k {tuple(x.shape)} does not match q {tuple(q.shape)}")
        if out is None:
            out = torch.empty_like(x)
            made.append(out)
        else:
            _cuda(out, "out_" + name, torch.bfloat16, 4, dev)
            if out.shape != x.shape:
                raise ValueError(f"out_{name} {tuple(out.shape)} does not match {tuple(x.shape)}")
        _written(out, "out_" + name)
        pairs.append((x.data_ptr(), _Strides(*_dims_last(x, name)), out.data_ptr(),
                      _Strides(*_dims_last(out, "out_" + name)), x.shape[1], out))
    with _On(dev, stream) as on:
        on.keep(*made)
        rc = lib.attn_rope(*pairs[0][:5], *pairs[1][:5], positions.data_ptr(), ps[0], ps[1] if B > 1 else 0,
                           positions.shape[0], table.data_ptr(), B, N, D, 2 * table.shape[0], 1 if adjacent else 0,
                           backward, on.handle)
    _done(rc, what)
    return pairs[0][5], pairs[1][5]


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

def _table(t, dev=None):
    _cuda(t, "table", torch.int32, 2, dev)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("table's last dim must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _int_outs(dev, want, out):
    """The int32 outputs by name: given ones checked, the others made."""
    got, made = {}, []
    unknown = set(out or ()) - set(want)
    if unknown:
        raise ValueError(f"unknown outputs {sorted(unknown)}")
    for name, n in want.items():
        t = (out or {}).get(name)
        if t is None:
            t = torch.empty(n, dtype=torch.int32, device=dev)
            made.append(t)
        else:
            _dense(t, name, torch.int32, 1, dev)
            if t.shape[0] != n:
                raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")
        got[name] = t
    return got, made


def _page_state(table, lens, arg, arg_name, free_pages, free_count):
    stride = _table(table)
    _written(table, "table")
    dev, B = table.device, table.shape[0]
    for t, name in ((lens, "lens"), (arg, arg_name)):
        _dense(t, name, torch.int32, 1, dev)
        if t.shape[0] != B:
            raise ValueError(f"{name} must have {B} elements (rows of table), got {t.shape[0]}")
    _dense(free_pages, "free_pages", torch.int32, 1, dev)
    _dense(free_count, "free_count", torch.int32, 1, dev)
    if free_count.shape[0] != 1:
        raise ValueError("free_count must have one element")
    return stride, dev, B


def attn_pages_assign(table, lens, new_lens, free_pages, free_count, page_size: int, max_tokens: int, out=None,
                      stream=None) -> dict:
    """Pages, slots and positions of ``new_lens`` further tokens of each request.

    All int32 on one device: ``table`` [B, max_pages] (updated in place),
    ``lens`` and ``new_lens`` [B], ``free_pages`` [capacity] and ``free_count``
    [1] (a stack of free page ids).  Returns a dict of lens [B], free_count
    [1], cu [B + 1], slots and positions [max_tokens], info [2] (info[0] != 0:
    the step was refused and nothing changed, see ATTN_PAGES_* in
    include/attn.h).  ``out`` may hold any of them; out["lens"] may be lens and
    out["free_count"] free_count, for updates in place."""
    stride, dev, B = _page_state(table, lens, new_lens, "new_lens", free_pages, free_count)
    o, made = _int_outs(dev, {"lens": B, "free_count": 1, "cu": B + 1, "slots": max_tokens, "positions": max_tokens,
                              "info": 2}, out)
    with _On(dev, stream) as on:
        on.keep(*made)
        rc = load_library().attn_pages_assign(
            table.data_ptr(), stride, table.shape[1], lens.data_ptr(), new_lens.data_ptr(), B, page_size,
            free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), o["lens"].data_ptr(),
            o["free_count"].data_ptr(), o["cu"].data_ptr(), o["slots"].data_ptr(), o["positions"].data_ptr(),
            max_tokens, o["info"].data_ptr(), on.handle)
    _done(rc, "attn_pages_assign")
    return o


def attn_pages_release(table, lens, keep_lens, free_pages, free_count, page_size: int, out=None, stream=None) -> dict:
    """Requests cut to ``keep_lens`` tokens (0: finished; negative: left alone),
    their pages back on the stack.  ``table`` and ``free_pages`` are updated in
    place; returns a dict of lens [B], free_count [1] and info [2]."""
    stride, dev, B = _page_state(table, lens, keep_lens, "keep_lens", free_pages, free_count)
    o, made = _int_outs(dev, {"lens": B, "free_count": 1, "info": 2}, out)
    with _On(dev, stream) as on:
        on.keep(*made)
        rc = load_library().attn_pages_release(
            table.data_ptr(), stride, table.shape[1], lens.data_ptr(), keep_lens.data_ptr(), B, page_size,
            free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), o["lens"].data_ptr(),
            o["free_count"].data_ptr(), o["info"].data_ptr(), on.handle)
    _done(rc, "attn_pages_release")
    return o


# ---------------------------------------------------------------- the 4-bit cache

def attn_kv4_page_bytes(head_dim: int, page_size: int) -> int:
    """Bytes of one page of one kv head."""
    n = int(load_library().attn_kv4_page_bytes(int(head_dim), int(page_size)))
    if n < 0:
        raise AttnError(n, "attn_kv4_page_bytes")
    return n


def attn_kv4_cache(num_pages: int, Hkv: int, head_dim: int, page_size: int, device="cuda") -> torch.Tensor:
    """An empty cache: uint8 [num_pages, Hkv, page bytes]."""
    return torch.zeros((num_pages, Hkv, attn_kv4_page_bytes(head_dim, page_size)), dtype=torch.uint8, device=device)


def _cache_dim(cache, page_size, dev=None):
    """Head dim of a cache: a page holds 72 bytes per token and group of 64 dims."""
    _dense(cache, "cache", torch.uint8, 3, dev)
    per = 72 * page_size
    if page_size < 1 or cache.shape[2] == 0 or cache.shape[2] % per:
        raise ValueError(f"cache {tuple(cache.shape)} is not one of pages of {page_size} tokens")
    return cache.shape[2] // per * _GROUP


def attn_kv4_append(k, v, slots, cache, page_size: int, stream=None) -> None:
    """Quantises k and v (bf16 [T, Hkv, D], any strides with a contiguous last
    dim) into the cache's slots (int32 [T]; -1 skips a token; no slot twice)."""
    D = _cache_dim(cache, page_size)
    dev = cache.device
    _cuda(k, "k", torch.bfloat16, 3, dev)
    _cuda(v, "v", torch.bfloat16, 3, dev)
    _dense(slots, "slots", torch.int32, 1, dev)
    T, H = slots.shape[0], cache.shape[1]
    if k.shape != v.shape or tuple(k.shape) != (T, H, D):
        raise ValueError(f"k {tuple(k.shape)} / v {tuple(v.shape)} do not match [{T}, {H}, {D}]")
    ks, vs = _dims_last(k, "k"), _dims_last(v, "v")
    with _On(dev, stream) as on:
        rc = load_library().attn_kv4_append(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slots.data_ptr(),
                                            cache.data_ptr(), cache.shape[0], T, H, D, page_size, on.handle)
    _done(rc, "attn_kv4_append")


def attn_kv4_read(slots, cache, page_size: int, out_k=None, out_v=None, stream=None):
    """K and V of the slots (int32 [T]) as bf16 [Hkv, T, D]: k[None], v[None]
    are attn_fwd's operands for a cached prefix.  Slot -1 reads as zeros."""
    D = _cache_dim(cache, page_size)
    dev = cache.device
    _dense(slots, "slots", torch.int32, 1, dev)
    T, H = slots.shape[0], cache.shape[1]
    made, outs = [], []
    for t, name in ((out_k, "out_k"), (out_v, "out_v")):
        if t is None:
            t = torch.empty((H, T, D), dtype=torch.bfloat16, device=dev)
            made.append(t)
        else:
            _cuda(t, name, torch.bfloat16, 3, dev)
            if tuple(t.shape) != (H, T, D):
                raise ValueError(f"{name} {tuple(t.shape)} does not match [{H}, {T}, {D}]")
            _written(t, name)
        outs.append(t)
    ks, vs = _dims_last(outs[0], "out_k"), _dims_last(outs[1], "out_v")
    with _On(dev, stream) as on:
        on.keep(*made)
        rc = load_library().attn_kv4_read(cache.data_ptr(), cache.shape[0], slots.data_ptr(), outs[0].data_ptr(), ks[0],
                                          ks[1], outs[1].data_ptr(), vs[0], vs[1], T, H, D, page_size, on.handle)
    _done(rc, "attn_kv4_read")
    return outs[0], outs[1]


def attn_fwd_kv4(q, cu, lens, table, cache, page_size: int, scale: float | None = None, causal: bool = True, out=None,
                 lse=None, stream=None):
    """O [T, Hq, D] (bf16), LSE [T, Hq] (fp32): attention of q (bf16 [T, Hq, D])
    over the cached tokens of each request.

    ``cu`` [B + 1], ``lens`` [B] and ``table`` [B, max_pages] int32 as
    attn_pages_assign gives them: request r has query tokens cu[r] .. cu[r+1] - 1
    and lens[r] cached tokens, theirs among them (``causal``: bottom-right
    aligned, as attn_fwd).  Rows outside cu[0] .. cu[B] are left as they were.
    Head dims 64, 128, 192, 256."""
    D = _cache_dim(cache, page_size)
    dev = cache.device
    _cuda(q, "q", torch.bfloat16, 3, dev)
    T, Hq = q.shape[0], q.shape[1]
    Hkv = cache.shape[1]
    if q.shape[2] != D:
        raise ValueError(f"q {tuple(q.shape)} does not match the cache's head dim {D}")
    stride = _table(table, dev)
    B = table.shape[0]
    _dense(cu, "cu", torch.int32, 1, dev)
    _dense(lens, "lens", torch.int32, 1, dev)
    if cu.shape[0] != B + 1 or lens.shape[0] != B:
        raise ValueError(f"cu {tuple(cu.shape)} / lens {tuple(lens.shape)} do not match {B} requests (rows of table)")
    made = []
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        made.append(out)
    else:
        _dense(out, "out", torch.bfloat16, 3, dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        made.append(lse)
    else:
        _dense(lse, "lse", torch.float32, 2, dev)
    if out.shape != q.shape or tuple(lse.shape) != (T, Hq):
        raise ValueError("out / lse shape mismatch")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    qs = _dims_last(q, "q")
    with _On(dev, stream) as on:
        on.keep(*made)
        rc = load_library().attn_fwd_kv4(q.data_ptr(), qs[0], qs[1], cu.data_ptr(), lens.data_ptr(), table.data_ptr(),
                                         stride, table.shape[1], cache.data_ptr(), cache.shape[0], out.data_ptr(),
                                         lse.data_ptr(), B, T, Hq, Hkv, D, page_size, scale, 1 if causal else 0,
                                         on.handle)
    _done(rc, "attn_fwd_kv4")
    return out, lse
