"""Torch-facing wrappers of the paged key-value cache of ``include/nf4.h``: new tokens written into
their pages, and attention of one new token a sequence over them.

As in ``ops``: PyTorch supplies device memory and the current stream, every step of the
computation runs in the library's kernels, and there is no CPU path.
"""
from __future__ import annotations

import functools
import struct
from typing import Optional

import torch

from . import _lib
from .block_ops import _DTYPES, _dtype, _fn, _on, _one_device, _raw_stream, _share_storage, _workspace5, _written

_CACHE = struct.Struct("@2P6qPqP2q5i4x")  # nf4_paged_cache


def _explain_cache(name, k_pages, v_pages, page_table, lengths, rows):
    """Why these are no cache with rows of its heads; rows: (what, tensor, heads or None)."""
    _one_device(name, k_pages, v_pages, page_table, lengths, *(t for _, t, _ in rows))
    _dtype(name, k_pages)
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or 0 in k_pages.shape[1:]:
        raise ValueError(f"{name}: k_pages and v_pages must be [pages, slots, heads, D] of one shape and dtype, got "
                         f"{tuple(k_pages.shape)} {k_pages.dtype} and {tuple(v_pages.shape)} {v_pages.dtype}")
    D = k_pages.shape[3]
    for what, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if D > 1 and t.stride(3) != 1:
            raise ValueError(f"{name}: {what} must have unit stride within a head")
    if lengths.dtype != torch.int32 or lengths.dim() != 1 or not lengths.is_contiguous():
        raise ValueError(f"{name}: lengths must be a contiguous int32 [sequences] tensor")
    if (page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != lengths.shape[0]
            or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError(f"{name}: page_table must be an int32 [{lengths.shape[0]}, pages of a sequence] tensor with unit column stride")
    for what, t, heads in rows:
        if t.dim() != 3 or t.dtype != k_pages.dtype or t.shape[2] != D or (heads is not None and t.shape[1] != heads):
            raise ValueError(f"{name}: {what} must be a {k_pages.dtype} [rows, {'heads' if heads is None else heads}, {D}] tensor, got "
                             f"{t.dtype} {tuple(t.shape)}")
        if D > 1 and t.stride(2) != 1:
            raise ValueError(f"{name}: {what} must have unit stride within a head")


def _cache(name, k_pages, v_pages, page_table, lengths, rows):
    """The packed nf4_paged_cache of checked arguments, and the cache's shape."""
    dt, dev, ks, kt, vt, ts, tt, ls = (k_pages.dtype, k_pages.device, k_pages.shape, k_pages.stride(), v_pages.stride(), page_table.shape,
                                       page_table.stride(), lengths.shape)
    at = k_pages.get_device()
    ok = (dt in _DTYPES and at >= 0 and len(ks) == 4 and v_pages.shape == ks and v_pages.dtype is dt and 0 not in ks[1:]
          and v_pages.get_device() == at and page_table.get_device() == at and lengths.get_device() == at
          and (kt[3] == 1 == vt[3] or ks[3] == 1) and lengths.dtype is torch.int32 and lengths.is_contiguous() and len(ls) == 1
          and page_table.dtype is torch.int32 and len(ts) == 2 and ts[0] == ls[0] and (tt[1] == 1 or ts[1] < 2))
    for _, t, heads in rows if ok else ():
        s = t.shape
        ok = (ok and t.dtype is dt and t.get_device() == at and len(s) == 3 and s[2] == ks[3] and (heads is None or s[1] == heads)
              and (t.stride(2) == 1 or s[2] == 1))
    if not ok:
        _explain_cache(name, k_pages, v_pages, page_table, lengths, rows)
        raise ValueError(f"{name}: arguments do not make a paged cache")
    pages, slots, Hk, D = ks
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), kt[0], kt[1], kt[2], vt[0], vt[1], vt[2], page_table.data_ptr(), tt[0],
                       lengths.data_ptr(), ls[0], pages, ts[1], slots, Hk, D, _DTYPES[dt]), dev, ls[0], Hk, D


def _refuse_grad(name, *ts):
    """The calls are seen by no autograd: a gradient that is asked for through them would be lost without a word."""
    if torch.is_grad_enabled() and any([t is not None and t.requires_grad for t in ts]):
        raise ValueError(f"{name} has no gradients: call it under torch.no_grad() or on detached tensors")


@functools.lru_cache(maxsize=1024)
def _slots_share(shape: tuple, stride: tuple) -> bool:
    """Whether rows of a tensor [..., D] may meet in memory (one dimension not inside another's steps)."""
    reach = shape[-1]
    for step, n in sorted((s, n) for s, n in zip(stride[:-1], shape[:-1]) if n > 1):
        if step < reach:
            return True
        reach += step * (n - 1)
    return False


@functools.lru_cache(maxsize=1024)
def _reach(shape: tuple, stride: tuple) -> int:
    """Values from a tensor's first to behind its last."""
    return 0 if 0 in shape else 1 + sum(s * (n - 1) for s, n in zip(stride, shape))


@functools.lru_cache(maxsize=1024)
def _meet(shape: tuple, one: tuple, other: tuple, apart: int) -> bool:
    """Whether rows of two tensors [..., D] of one shape, the second's first value `apart` behind the first's, may meet in
    memory."""
    if 0 in shape or apart >= _reach(shape, one) or -apart >= _reach(shape, other):
        return False
    steps = sorted(((s, t, n) for s, t, n in zip(one[:-1], other[:-1], shape[:-1]) if n > 1), reverse=True)
    if any(s != t for s, t, _ in steps) or _slots_share(shape, one):
        return True

    def hit(rest, steps):  # inner dimensions reach less than a step, so two counts of it can meet `rest`
        if not steps:
            return abs(rest) < shape[-1]
        s, _, n = steps[0]
        return any(hit(rest - i * s, steps[1:]) for i in (rest // s, rest // s + 1) if abs(i) < n)

    return hit(apart, steps)


@functools.lru_cache(maxsize=1024)
def _writable(shape: tuple, k: tuple, v: tuple, apart: int) -> bool:
    """Whether every slot of key and value pages of these strides has memory of its own."""
    return not (_slots_share(shape, k) or _slots_share(shape, v) or _meet(shape, k, v, apart))


def _check_out(name, out, q, k_pages, v_pages):
    """out: q itself, or memory of its own."""
    shape, to, tq, e = q.shape, out.stride(), q.stride(), q.element_size()
    if out.shape != shape or _share_storage(out):
        raise ValueError(f"{name}: out must have q's shape, and rows that do not share storage")
    at = out.data_ptr()
    apart, end = (at - q.data_ptr()) // e, at + e * _reach(shape, to)
    itself = apart == 0 and (to == tq or all(s == t for s, t, n in zip(to, tq, shape) if n > 1))
    meets = not itself and _meet(shape, tq, to, apart)
    for p in (k_pages, v_pages):
        first = p.data_ptr()
        meets = meets or (first < end and at < first + e * _reach(p.shape, p.stride()))
    if meets:
        raise ValueError(f"{name}: out must be q itself or share no storage with q and the pages")


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                 lengths: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None) -> None:
    """nf4_paged_append: writes new tokens' rows k, v [T, Hk, D] into the pages [pages, slots, Hk, D] (any strides whose
    slots share no storage, keys and values neither: a transposed view of [pages, Hk, slots, D] will do, and so will two halves
    of one buffer).  k and v may not lie in slots that the call writes.  Token t of sequence i lies in page
    page_table[i, t // slots], slot t % slots.  `lengths` int32 [sequences] counts the new tokens already: rows
    cu_seqlens[i] .. cu_seqlens[i + 1] - 1 are the last tokens of sequence i (a prompt or a chunk of one); without
    cu_seqlens row i is the newest token of sequence i.  Rows of sequences of length 0, and rows whose page is missing
    from the table or lies past its last column (recorded in the device status), are not written.  No gradients, as in
    paged_attention."""
    name = "paged_append"
    Hk = k_pages.shape[2] if k_pages.dim() == 4 else -1
    d, dev, n, _, _ = _cache(name, k_pages, v_pages, page_table, lengths, (("k", k, Hk), ("v", v, Hk)))
    _refuse_grad(name, k, v, k_pages, v_pages)
    T, cu = k.shape[0], None
    if v.shape[0] != T or (cu_seqlens is None and T != n):
        raise ValueError(f"{name}: {T} and {v.shape[0]} rows of keys and values for {n} sequences")
    if cu_seqlens is not None:
        cu = cu_seqlens.data_ptr()
        if (cu_seqlens.dtype is not torch.int32 or cu_seqlens.shape != (n + 1,) or not cu_seqlens.is_contiguous()
                or cu_seqlens.device != dev):
            raise ValueError(f"{name}: cu_seqlens must be a contiguous int32 [{n + 1}] tensor on {dev}")
    if not _writable(k_pages.shape, k_pages.stride(), v_pages.stride(), (v_pages.data_ptr() - k_pages.data_ptr()) // k_pages.element_size()):
        raise ValueError(f"{name}: slots of the pages share storage")
    kt, vt = k.stride(), v.stride()
    with _on(dev):
        rc = _fn("nf4_paged_append")(d, k.data_ptr(), kt[0], kt[1], v.data_ptr(), vt[0], vt[1], cu, T, _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_paged_append")
    _written((k_pages, v_pages))


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None):
    """nf4_paged_attention: attention of one query token a sequence, q [sequences, Hq, D] (any sequence and head strides),
    over the lengths[i] tokens that page_table names for it (pages and table as in paged_append; the new token's own
    keys and values are appended first).  Query head h reads key head h // (Hq // Hk); `scale` defaults to D ** -0.5.
    Returns (o [sequences, Hq, D], lse fp32 [sequences, Hq]); a sequence of length 0 gives zeros and -inf.  `out` takes o in
    place of a new tensor: q itself, or any strides whose rows share no storage with each other, q or the pages.  Tables and lengths are read on
    the device, so a captured graph follows them.  No gradients: with gradients enabled, tensors that require one are refused."""
    name = "paged_attention"
    d, dev, n, Hk, D = _cache(name, k_pages, v_pages, page_table, lengths, (("q", q, None),) if out is None else (("q", q, None), ("out", out, None)))
    _refuse_grad(name, q, k_pages, v_pages, out)
    Hq = q.shape[1]
    if q.shape[0] != n or Hq == 0 or Hq % Hk:
        raise ValueError(f"{name}: q {tuple(q.shape)} does not fit {n} sequences of {Hk} key heads")
    if out is not None:
        _check_out(name, out, q, k_pages, v_pages)
    o = torch.empty((n, Hq, D), dtype=q.dtype, device=dev) if out is None else out
    lse = torch.empty((n, Hq), dtype=torch.float32, device=dev)
    qt, ot = q.stride(), o.stride()
    with _on(dev):
        need = _workspace5(_lib.OP_PAGED_ATTENTION, 0, Hq, D, Hk, dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        rc = _fn("nf4_paged_attention")(d, q.data_ptr(), qt[0], qt[1], Hq, D ** -0.5 if scale is None else scale, o.data_ptr(), ot[0],
                                        ot[1], lse.data_ptr(), ws.data_ptr(), need, _raw_stream(dev))
    if rc:
        _lib.check(rc, "nf4_paged_attention")
    if out is not None:
        _written((out,))
    return o, lse
