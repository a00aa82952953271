"""Pages of a paged cache: who holds them, their copies, and compaction.

A ``PagePool`` says on the device which pages each sequence holds and how many
sequences hold each page. ``pages_resize`` gives a sequence pages for more
tokens or takes them back, ``pages_fork`` continues one sequence as several that
share its full pages; both return the pages to be copied, which
``kv_copy_pages`` does in all layers' caches at once (a ``cache_group``).
``kv_compact`` keeps the tokens of an accepted path after verification.

Argument marshalling only, as in ``w4a16``: shapes, types and devices are checked
here, sizes and alignment again in the library. Calls enqueue on the current
stream of the tensors' device and never synchronise, so that they can be
captured into a graph; there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import struct
from typing import NamedTuple, Sequence

import torch

from . import w4a16 as _W
from .attn import _CACHE, KVCache, _array, _call, _packed_cache

MAX_LIST = 4096
_FIELDS = struct.Struct("@" + _CACHE)
_PAGES = struct.Struct("@PPPqqiiiiPPPPPii")
_COPY = struct.Struct("@PPPqii")
_COMPACT = struct.Struct("@PPPPPPPqiiii")


class PagePool(NamedTuple):
    """``refs`` int32 ``[pages]``: how many sequences hold each page; ``block_table``
    int32 ``[rows, table_pages]`` and ``lens`` int32 ``[rows]``: the pages and tokens
    of each sequence, entries behind its pages -1. ``tree_attention`` takes the
    table and lengths as they are."""
    refs: torch.Tensor
    block_table: torch.Tensor
    lens: torch.Tensor
    page_size: int


class CacheGroup(NamedTuple):
    """Caches of one geometry (a model's layers), checked once, as the library takes them; ``apart``:
    no two of their arrays share memory."""
    caches: tuple[KVCache, ...]
    fields: ctypes.Array
    apart: bool = True


def page_pool(pages: int, rows: int, table_pages: int, page_size: int = 64, device="cuda") -> PagePool:
    """A pool in which every page is free and every sequence empty."""
    return PagePool(torch.zeros(pages, dtype=torch.int32, device=device),
                    torch.full((rows, table_pages), -1, dtype=torch.int32, device=device),
                    torch.zeros(rows, dtype=torch.int32, device=device), page_size)


def _apart(addresses: tuple[int, ...], nbytes: int) -> bool:
    """Whether arrays of that many bytes at the addresses lie beside each other."""
    addresses = sorted(addresses)
    return nbytes == 0 or min(map(operator.sub, addresses[1:], addresses)) >= nbytes


def _packed(caches: Sequence[KVCache]) -> tuple[tuple[KVCache, ...], list[tuple]]:
    """The caches and their fields, checked but for where they lie."""
    caches = tuple(KVCache(*c) for c in caches)
    if not caches:
        raise ValueError("a group needs a cache")
    dev = caches[0].k.device
    if dev.type != "cuda":
        raise ValueError("all tensors must be on the same GPU")
    fields = [_packed_cache(c, dev) for c in caches]
    if any(f[4:] != fields[0][4:] or c.k.dtype != caches[0].k.dtype for f, c in zip(fields, caches)):
        raise ValueError("the caches of a group must have one shape and dtype")
    return caches, fields


def _group(caches: tuple[KVCache, ...], fields: list[tuple], apart: bool = True) -> CacheGroup:
    held = b"".join(_FIELDS.pack(*f) for f in fields)
    return CacheGroup(caches, (ctypes.c_char * len(held)).from_buffer_copy(held), apart)


def cache_group(caches: Sequence[KVCache]) -> CacheGroup:
    """The given caches (at least one, on one GPU, alike but for their memory) as a group."""
    caches, fields = _packed(caches)
    k, v, k_scale, v_scale, *_ = zip(*fields)
    one = caches[0]
    return _group(caches, fields, _apart(k + v, one.k.numel() * one.k.element_size()) and (
        one.k_scale is None or _apart(k_scale + v_scale, one.k_scale.numel() * 4)))


def _pool(pool: PagePool, dev) -> tuple:
    refs, table, lens, size = pool
    if refs.dim() != 1 or table.dim() != 2 or lens.dim() != 1:
        raise ValueError("a pool has refs [pages], block_table [rows, table_pages] and lens [rows]")
    rows, entries = table.shape
    stride, one = table.stride()
    if table.dtype != torch.int32 or table.device != dev or (one != 1 and entries > 1):
        raise ValueError("block_table must be int32 [rows, table_pages] on one GPU, its last dimension contiguous")
    if rows <= 1:
        stride = entries                    # no other row to go to
    return (_array(refs, "refs", torch.int32, dev, refs.shape[0]), table.data_ptr(),
            _array(lens, "lens", torch.int32, dev, rows), refs.shape[0], stride, rows, entries, size, 0)


def _change(fn, pool, first, second, names):
    if not pool.refs.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    dev = pool.refs.device
    fields = _pool(pool, dev)
    if first.dim() != 1:
        raise ValueError(f"{names[0]} must be int32, 1-D")
    n = first.shape[0]
    lists = _array(first, names[0], torch.int32, dev, n), _array(second, names[1], torch.int32, dev, n)
    out = first.new_empty((3, n))
    served, src, dst = torch.unbind(out)
    at = out.data_ptr()
    _call(fn, dev, _PAGES.pack(*fields, *lists, at, at + 4 * n, at + 8 * n, n, 0))
    return served, src, dst


def pages_resize(pool: PagePool, rows: torch.Tensor,
                 lens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gives the sequences ``rows`` (int32 ``[n]``, up to 4096) pages for ``lens`` (int32
    ``[n]``) tokens, or takes back those behind; a length of 0 frees a sequence. A page
    that the next token would be written to and that others hold too is replaced by one of
    the sequence's own. Returns ``(served, src, dst)``, int32 ``[n]``: 1 for the
    rows that changed, 0 for those refused (outside the pool, listed before, too long, or no pages left, from
    the first for which there are too few on), and the pages that ``kv_copy_pages`` has to copy, -1 for
    none. Pages that this call takes back are given out by later ones."""
    return _change(_W.lib().w4a16_pages_resize, pool, rows, lens, ("rows", "lens"))


def pages_fork(pool: PagePool, parents: torch.Tensor,
               children: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Continues the sequences ``parents`` (int32 ``[n]``, up to 4096) as the empty
    rows ``children`` (int32 ``[n]``) too: full pages are shared, a partly filled last
    one gets a copy. Returns ``(served, src, dst)`` as ``pages_resize``; refused are
    children that hold tokens or are listed before."""
    return _change(_W.lib().w4a16_pages_fork, pool, parents, children, ("parents", "children"))


def kv_copy_pages(group: CacheGroup, src: torch.Tensor, dst: torch.Tensor) -> None:
    """Copies page ``src[i]`` to ``dst[i]`` (int32 ``[n]``) in every cache of the group, scales
    included; pairs with a page outside it, such as -1, are skipped. No page
    is written twice, or read and written."""
    dev = group.caches[0].k.device
    if src.dim() != 1:
        raise ValueError("src must be int32, 1-D")
    n = src.shape[0]
    lists = _array(src, "src", torch.int32, dev, n), _array(dst, "dst", torch.int32, dev, n)
    _call(_W.lib().w4a16_kv_copy_pages, dev,
          _COPY.pack(ctypes.addressof(group.fields), *lists, n, len(group.caches), 0))


def kv_compact(group: CacheGroup, block_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
               path: torch.Tensor, counts: torch.Tensor) -> torch.Tensor:
    """Keeps the accepted ones of each sequence's new tokens, the last
    ``q_starts[b + 1] - q_starts[b]`` of ``kv_lens[b]``: those that ``path`` (int32
    ``[sequences, width]``, ascending) names in its first ``counts[b]`` (int32) entries, as
    ``scoring.verify_drafts`` returns them, move to the front of the new ones in every
    cache of the group, whose arrays have to lie apart. Returns the new lengths, int32 ``[sequences]``.
    ``block_table``, ``kv_lens`` and ``q_starts`` as for ``tree_attention``, with a row for each sequence and its new
    tokens in pages that no other holds (as ``pages_resize`` leaves them)."""
    if not group.apart:
        raise ValueError("arrays of the group's caches share memory, where tokens would move twice")
    dev = group.caches[0].k.device
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.device != dev:
        raise ValueError("block_table must be int32 [sequences, pages] on the caches' device")
    B, entries = block_table.shape
    row, one = block_table.stride()
    if one != 1 and entries > 1:
        raise ValueError("block_table: the last dimension must be contiguous")
    if B <= 1:
        row = entries                       # no other row to go to
    if path.dim() != 2:
        raise ValueError("path must be int32 [sequences, width]")
    width = path.shape[1]
    new = torch.empty_like(kv_lens, memory_format=torch.contiguous_format)
    _call(_W.lib().w4a16_kv_compact, dev,
          _COMPACT.pack(ctypes.addressof(group.fields), block_table.data_ptr(),
                        _array(kv_lens, "kv_lens", torch.int32, dev, B),
                        _array(q_starts, "q_starts", torch.int32, dev, B + 1),
                        _array(path, "path", torch.int32, dev, B, width),
                        _array(counts, "counts", torch.int32, dev, B), new.data_ptr(), row, B, entries, width,
                        len(group.caches)))
    return new
