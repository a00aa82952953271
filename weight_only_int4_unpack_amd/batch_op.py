"""Verification of drafts, pages of the cache and adapters as opaque torch operators.

``torch.ops.w4a16.verify_drafts``, ``pages_resize``, ``pages_fork``,
``kv_copy_pages``, ``kv_compact``, ``lora_plan`` and ``lora``: as for the
operators of ``serve_op``, a graph compiler sees one call node each, and how
the work is split is chosen on every call from the runtime sizes. The pool's
arrays are written by ``pages_resize`` and ``pages_fork``, the caches by
``kv_copy_pages`` and ``kv_compact``, as their schemas say; the others return
new tensors. The fake implementations give shapes, dtypes and devices and apply
the checks that need no data. The functions of the same names here are facades
with the signatures of ``scoring``, ``paging`` and ``adapters`` (without their
output arguments).
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import adapters as _L
from . import attn as _A
from . import paging as _P
from . import scoring as _S
from .serve_op import _FLOATS, _check_cache, _check_list, _need


@torch.library.custom_op("w4a16::verify_drafts", mutates_args=())
def _verify_op(logits: torch.Tensor, ids: torch.Tensor, q_starts: torch.Tensor, max_q: int,
               uniforms: torch.Tensor, final_uniforms: torch.Tensor, parents: torch.Tensor | None = None,
               draft_probs: torch.Tensor | None = None, temperatures: torch.Tensor | None = None
               ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return _S.verify_drafts(logits, ids, q_starts, max_q, uniforms, final_uniforms, parents, draft_probs,
                            temperatures)


@_verify_op.register_fake
def _verify_fake(logits, ids, q_starts, max_q, uniforms, final_uniforms, parents=None, draft_probs=None,
                 temperatures=None):
    _need(logits.dim() == 2 and logits.dtype in (*_FLOATS, torch.float32),
          "logits must be float16, bfloat16 or float32 [tokens, vocab]")
    _need(q_starts.dim() == 1 and q_starts.dtype == torch.int32, "q_starts must be int32 [sequences + 1]")
    T, B = logits.shape[0], q_starts.shape[0] - 1
    _check_list(ids, "ids", torch.int64, T)
    _check_list(uniforms, "uniforms", torch.float32, T)
    _check_list(final_uniforms, "final_uniforms", torch.float32, B)
    _need(parents is None or draft_probs is None, "draft_probs go with chains: parents must be None")
    if parents is not None:
        _check_list(parents, "parents", torch.int32, T)
    if draft_probs is not None:
        _check_list(draft_probs, "draft_probs", torch.float32, *logits.shape)
    if temperatures is not None:
        _check_list(temperatures, "temperatures", torch.float32, B)
    return ids.new_empty((B, max_q)), q_starts.new_empty((B, max_q)), q_starts.new_empty((B,))


def verify_drafts(logits: torch.Tensor, ids: torch.Tensor, q_starts: torch.Tensor, max_q: int,
                  uniforms: torch.Tensor, final_uniforms: torch.Tensor,
                  parents: torch.Tensor | None = None, draft_probs: torch.Tensor | None = None,
                  temperatures: torch.Tensor | None = None
                  ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``scoring.verify_drafts`` through ``torch.ops.w4a16.verify_drafts``."""
    return torch.ops.w4a16.verify_drafts(logits, ids, q_starts, max_q, uniforms, final_uniforms, parents,
                                         draft_probs, temperatures)


def _check_pool(refs, block_table, lens):
    _need(refs.dim() == 1 and refs.dtype == torch.int32, "refs must be int32 [pages]")
    _need(block_table.dim() == 2 and block_table.dtype == torch.int32,
          "block_table must be int32 [rows, table_pages]")
    _check_list(lens, "lens", torch.int32, block_table.shape[0])


def _change_fake(first, second, names):
    _need(first.dim() == 1 and first.dtype == torch.int32, f"{names[0]} must be int32, 1-D")
    _check_list(second, names[1], torch.int32, first.shape[0])
    return tuple(torch.empty_like(first) for _ in range(3))


def _apart(out):
    """The rows of one array as tensors of their own, as an operator has to return them."""
    return tuple(x.clone() for x in out)


@torch.library.custom_op("w4a16::pages_resize", mutates_args=("refs", "block_table", "pool_lens"))
def _resize_op(refs: torch.Tensor, block_table: torch.Tensor, pool_lens: torch.Tensor, page_size: int,
               rows: torch.Tensor, lens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return _apart(_P.pages_resize(_P.PagePool(refs, block_table, pool_lens, page_size), rows, lens))


@_resize_op.register_fake
def _resize_fake(refs, block_table, pool_lens, page_size, rows, lens):
    _check_pool(refs, block_table, pool_lens)
    return _change_fake(rows, lens, ("rows", "lens"))


def pages_resize(pool: _P.PagePool, rows: torch.Tensor,
                 lens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``paging.pages_resize`` through ``torch.ops.w4a16.pages_resize``."""
    return torch.ops.w4a16.pages_resize(*pool, rows, lens)


@torch.library.custom_op("w4a16::pages_fork", mutates_args=("refs", "block_table", "pool_lens"))
def _fork_op(refs: torch.Tensor, block_table: torch.Tensor, pool_lens: torch.Tensor, page_size: int,
             parents: torch.Tensor, children: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return _apart(_P.pages_fork(_P.PagePool(refs, block_table, pool_lens, page_size), parents, children))


@_fork_op.register_fake
def _fork_fake(refs, block_table, pool_lens, page_size, parents, children):
    _check_pool(refs, block_table, pool_lens)
    return _change_fake(parents, children, ("parents", "children"))


def pages_fork(pool: _P.PagePool, parents: torch.Tensor,
               children: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``paging.pages_fork`` through ``torch.ops.w4a16.pages_fork``."""
    return torch.ops.w4a16.pages_fork(*pool, parents, children)


def _lists(group: _P.CacheGroup):
    """The group's tensors by kind; without scales those lists are empty."""
    k, v, ks, vs = zip(*group.caches)
    return (list(k), list(v), *([] if ks[0] is None else list(s) for s in (ks, vs)))


def _caches(k, v, k_scales, v_scales) -> list[_A.KVCache]:
    none = [None] * len(k)
    return list(map(_A.KVCache, k, v, k_scales or none, v_scales or none))


def _check_group(k, v, k_scales, v_scales):
    n = len(k)
    _need(n > 0 and len(v) == n and len(k_scales) == len(v_scales) and len(k_scales) in (0, n),
          "a group has as many k as v, and scales for each or none")
    none = [None] * n
    for c in zip(k, v, k_scales or none, v_scales or none):
        _check_cache(*c, c[0].dtype)
        _need(c[0].shape == k[0].shape and c[0].dtype == k[0].dtype,
              "the caches of a group must have one shape and dtype")


@torch.library.custom_op("w4a16::kv_copy_pages", mutates_args=("k", "v", "k_scales", "v_scales"))
def _copy_op(k: Sequence[torch.Tensor], v: Sequence[torch.Tensor], k_scales: Sequence[torch.Tensor],
             v_scales: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor) -> None:
    # (a copy does not ask whether the caches lie apart)
    _P.kv_copy_pages(_P._group(*_P._packed(_caches(k, v, k_scales, v_scales))), src, dst)


@_copy_op.register_fake
def _copy_fake(k, v, k_scales, v_scales, src, dst):
    _check_group(k, v, k_scales, v_scales)
    _need(src.dim() == 1 and src.dtype == torch.int32, "src must be int32, 1-D")
    _check_list(dst, "dst", torch.int32, src.shape[0])


def kv_copy_pages(group: _P.CacheGroup, src: torch.Tensor, dst: torch.Tensor) -> None:
    """``paging.kv_copy_pages`` through ``torch.ops.w4a16.kv_copy_pages``."""
    torch.ops.w4a16.kv_copy_pages(*_lists(group), src, dst)


@torch.library.custom_op("w4a16::kv_compact", mutates_args=("k", "v", "k_scales", "v_scales"))
def _compact_op(k: Sequence[torch.Tensor], v: Sequence[torch.Tensor], k_scales: Sequence[torch.Tensor],
                v_scales: Sequence[torch.Tensor], block_table: torch.Tensor, kv_lens: torch.Tensor,
                q_starts: torch.Tensor, path: torch.Tensor, counts: torch.Tensor) -> torch.Tensor:
    return _P.kv_compact(_P.cache_group(_caches(k, v, k_scales, v_scales)), block_table, kv_lens, q_starts, path, counts)


@_compact_op.register_fake
def _compact_fake(k, v, k_scales, v_scales, block_table, kv_lens, q_starts, path, counts):
    _check_group(k, v, k_scales, v_scales)
    _need(block_table.dim() == 2 and block_table.dtype == torch.int32,
          "block_table must be int32 [sequences, pages]")
    B = block_table.shape[0]
    _check_list(kv_lens, "kv_lens", torch.int32, B)
    _check_list(q_starts, "q_starts", torch.int32, B + 1)
    _need(path.dim() == 2, "path must be int32 [sequences, width]")
    _check_list(path, "path", torch.int32, B, path.shape[1])
    _check_list(counts, "counts", torch.int32, B)
    return torch.empty_like(kv_lens, memory_format=torch.contiguous_format)


def kv_compact(group: _P.CacheGroup, block_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
               path: torch.Tensor, counts: torch.Tensor) -> torch.Tensor:
    """``paging.kv_compact`` through ``torch.ops.w4a16.kv_compact``."""
    return torch.ops.w4a16.kv_compact(*_lists(group), block_table, kv_lens, q_starts, path, counts)


def _plan_room(tokens, adapters):
    """Bytes that hold a plan with tiles of 16 or of 64 tokens, in a form that symbolic sizes go
    through: tiles are at most ceil(tokens / rows) + adapters, of 4 (1 + rows) bytes, and 16."""
    return 16 + 272 * ((tokens + 63) // 64 + adapters)


@torch.library.custom_op("w4a16::lora_plan", mutates_args=())
def _plan_op(index: torch.Tensor, adapters: int) -> torch.Tensor:
    return _L.lora_plan(index, adapters, _plan_room(index.shape[0], adapters)).data


@_plan_op.register_fake
def _plan_fake(index, adapters):
    _need(index.dim() == 1 and index.dtype == torch.int32, "index must be int32 [tokens]")
    return index.new_empty((_plan_room(index.shape[0], adapters),), dtype=torch.uint8)


def lora_plan(index: torch.Tensor, adapters: int) -> _L.LoraPlan:
    """``adapters.lora_plan`` through ``torch.ops.w4a16.lora_plan``."""
    return _L.LoraPlan(torch.ops.w4a16.lora_plan(index, adapters), index.shape[0], adapters)


@torch.library.custom_op("w4a16::lora", mutates_args=())
def _lora_op(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, plan: torch.Tensor,
             base: torch.Tensor | None = None, scales: torch.Tensor | None = None,
             ranks: torch.Tensor | None = None, plan_tokens: int | None = None,
             plan_adapters: int | None = None) -> torch.Tensor:
    return _L.lora(x, a, b, _L.LoraPlan(plan, x.shape[0] if plan_tokens is None else plan_tokens,
                                        a.shape[0] if plan_adapters is None else plan_adapters), base, scales, ranks)


@_lora_op.register_fake
def _lora_fake(x, a, b, plan, base=None, scales=None, ranks=None, plan_tokens=None, plan_adapters=None):
    _need(x.dim() == 2 and a.dim() == 3 and b.dim() == 3,
          "x must be [tokens, k], a [adapters, rank, k], b [adapters, n, rank]")
    _need(x.dtype in _FLOATS, "x must be float16 or bfloat16")
    R, rank, N = a.shape[0], a.shape[1], b.shape[1]
    _check_list(a, "a", x.dtype, R, rank, x.shape[1])
    _check_list(b, "b", x.dtype, R, N, rank)
    _need(plan.dim() == 1 and plan.dtype == torch.uint8, "plan must be lora_plan's")
    _need((plan_tokens is None or plan_tokens == x.shape[0]) and (plan_adapters is None or plan_adapters == R),
          f"the plan is for {plan_tokens} tokens and {plan_adapters} adapters, not {x.shape[0]} and {R}")
    if base is not None:
        _check_list(base, "base", x.dtype, x.shape[0], N)
    if scales is not None:
        _check_list(scales, "scales", torch.float32, R)
    if ranks is not None:
        _check_list(ranks, "ranks", torch.int32, R)
    return x.new_empty((x.shape[0], N))


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, plan: _L.LoraPlan,
         base: torch.Tensor | None = None, scales: torch.Tensor | None = None,
         ranks: torch.Tensor | None = None) -> torch.Tensor:
    """``adapters.lora`` through ``torch.ops.w4a16.lora``, which sees the plan's memory alone and is told
    what it is for (``plan_tokens``, ``plan_adapters``; a call without them vouches for x's and a's)."""
    return torch.ops.w4a16.lora(x, a, b, plan.data, base, scales, ranks, plan.tokens, plan.adapters)
