"""Rotation, cache, attention and scoring as opaque torch operators.

``torch.ops.w4a16.rope``, ``kv_write``, ``kv_read``, ``tree_attention`` and
``token_logprobs``: as for ``torch.ops.w4a16.gemm``, a graph compiler sees one
call node each, and how the work is split is chosen on every call from the
runtime sizes. ``kv_write`` alone writes an input, the cache, and says so in
its schema; the others return new tensors. The fake implementations give
shapes, dtypes and devices and apply the checks that need no data, so a
malformed call fails while tracing. The functions of the same names here are
facades with the signatures of ``attn`` and ``scoring`` (without their output
arguments).
"""
from __future__ import annotations

import math

import torch

from . import attn as _A
from . import scoring as _S

_FLOATS = (torch.float16, torch.bfloat16)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _check_heads(x, what):
    _need(x.dim() == 3 and x.dtype in _FLOATS,
          f"{what} must be float16 or bfloat16 [tokens, heads, head_dim]")


def _check_cache(k_cache, v_cache, k_scale, v_scale, dtype):
    _need(k_cache.dim() == 4 and k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype,
          "the cache's k and v must be [pages, heads, page_size, head_dim] alike")
    if k_cache.dtype in (torch.float8_e4m3fn, torch.int8):
        _need(k_scale is not None and v_scale is not None, "a quantised cache needs k_scale and v_scale")
        for s in (k_scale, v_scale):
            _need(s.dtype == torch.float32 and s.shape == k_cache.shape[:3],
                  "scales must be float32 [pages, heads, page_size]")
    else:
        _need(k_cache.dtype == dtype, "a 16-bit cache must have the tokens' dtype")
        _need(k_scale is None and v_scale is None, "a 16-bit cache has no scales")


def _check_list(x, what, dtype, *shape):
    _need(x.dtype == dtype and x.dim() == len(shape) and tuple(x.shape) == shape,
          f"{what} must be {dtype} {list(shape)}")


def _check_table(table, head_dim):
    _need(table.dim() == 2 and table.dtype == torch.float32 and table.shape[1] <= head_dim,
          "table must be float32 [positions, rot_dim]")


@torch.library.custom_op("w4a16::rope", mutates_args=())
def _rope_op(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
             interleaved: bool = False, inverse: bool = False) -> torch.Tensor:
    return _A.rope(x, positions, table, interleaved, inverse)


@_rope_op.register_fake
def _rope_fake(x, positions, table, interleaved=False, inverse=False):
    _check_heads(x, "x")
    _check_list(positions, "positions", torch.int64, x.shape[0])
    _check_table(table, x.shape[2])
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
         interleaved: bool = False, inverse: bool = False) -> torch.Tensor:
    """``attn.rope`` through ``torch.ops.w4a16.rope``."""
    return torch.ops.w4a16.rope(x, positions, table, interleaved, inverse)


@torch.library.custom_op("w4a16::kv_write",
                         mutates_args=("k_cache", "v_cache", "k_scale", "v_scale"))
def _kv_write_op(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, k_scale: torch.Tensor | None, v_scale: torch.Tensor | None,
                 positions: torch.Tensor | None = None, table: torch.Tensor | None = None,
                 interleaved: bool = False, q: torch.Tensor | None = None) -> torch.Tensor:
    out = _A.kv_write(k, v, slots, _A.KVCache(k_cache, v_cache, k_scale, v_scale), positions, table,
                      interleaved, q)
    return k.new_empty((0,)) if out is None else out


@_kv_write_op.register_fake
def _kv_write_fake(k, v, slots, k_cache, v_cache, k_scale, v_scale, positions=None, table=None,
                   interleaved=False, q=None):
    _check_heads(k, "k")
    _need(v.shape == k.shape and v.dtype == k.dtype, "k and v must have one shape and dtype")
    _check_cache(k_cache, v_cache, k_scale, v_scale, k.dtype)
    _need(k_cache.shape[1] == k.shape[1] and k_cache.shape[3] == k.shape[2],
          "the cache must hold k's heads")
    _check_list(slots, "slots", torch.int64, k.shape[0])
    _need((positions is None) == (table is None), "positions and table go together")
    if table is not None:
        _check_list(positions, "positions", torch.int64, k.shape[0])
        _check_table(table, k.shape[2])
    if q is None:
        return k.new_empty((0,))
    _need(table is not None, "q is given to be rotated: positions and table are needed")
    _check_heads(q, "q")
    _need(q.dtype == k.dtype and q.shape[0] == k.shape[0] and q.shape[2] == k.shape[2],
          "q must be [tokens, q_heads, head_dim] like k")
    return torch.empty_like(q, memory_format=torch.contiguous_format)


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: _A.KVCache,
             positions: torch.Tensor | None = None, table: torch.Tensor | None = None,
             interleaved: bool = False, q: torch.Tensor | None = None) -> torch.Tensor | None:
    """``attn.kv_write`` through ``torch.ops.w4a16.kv_write``."""
    out = torch.ops.w4a16.kv_write(k, v, slots, *cache, positions, table, interleaved, q)
    return None if q is None else out


@torch.library.custom_op("w4a16::kv_read", mutates_args=())
def _kv_read_op(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor | None,
                v_scale: torch.Tensor | None, slots: torch.Tensor,
                dtype: torch.dtype) -> tuple[torch.Tensor, torch.Tensor]:
    return _A.kv_read(_A.KVCache(k_cache, v_cache, k_scale, v_scale), slots, dtype)


@_kv_read_op.register_fake
def _kv_read_fake(k_cache, v_cache, k_scale, v_scale, slots, dtype):
    _need(dtype in _FLOATS, "dtype must be float16 or bfloat16")
    _check_cache(k_cache, v_cache, k_scale, v_scale, dtype)
    _need(slots.dim() == 1 and slots.dtype == torch.int64, "slots must be int64, 1-D")
    shape = (slots.shape[0], k_cache.shape[1], k_cache.shape[3])
    return k_cache.new_empty(shape, dtype=dtype), k_cache.new_empty(shape, dtype=dtype)


def kv_read(cache: _A.KVCache, slots: torch.Tensor,
            dtype: torch.dtype | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """``attn.kv_read`` through ``torch.ops.w4a16.kv_read``."""
    if dtype is None:
        dtype = cache.k.dtype if cache.k.dtype in _FLOATS else torch.bfloat16
    return torch.ops.w4a16.kv_read(*cache, slots, dtype)


@torch.library.custom_op("w4a16::tree_attention", mutates_args=())
def _tree_attention_op(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scale: torch.Tensor | None, v_scale: torch.Tensor | None,
                       block_table: torch.Tensor, kv_lens: torch.Tensor, q_starts: torch.Tensor,
                       max_q: int, mask: torch.Tensor | None,
                       scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    return _A.tree_attention(q, _A.KVCache(k_cache, v_cache, k_scale, v_scale), block_table, kv_lens,
                             q_starts, max_q, mask, scale)


@_tree_attention_op.register_fake
def _tree_attention_fake(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q_starts,
                         max_q, mask, scale):
    _check_heads(q, "q")
    _check_cache(k_cache, v_cache, k_scale, v_scale, q.dtype)
    _need(k_cache.shape[3] == q.shape[2] and q.shape[1] % k_cache.shape[1] == 0,
          "the cache's heads must divide q's and have its head_dim")
    _need(block_table.dim() == 2 and block_table.dtype == torch.int32,
          "block_table must be int32 [sequences, pages]")
    _check_list(kv_lens, "kv_lens", torch.int32, block_table.shape[0])
    _check_list(q_starts, "q_starts", torch.int32, block_table.shape[0] + 1)
    if mask is not None:
        _need(mask.dim() == 2 and mask.dtype == torch.int64 and mask.shape[0] == q.shape[0],
              "mask must be int64 [tokens, words]")
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            q.new_empty(q.shape[:2], dtype=torch.float32))


def tree_attention(q: torch.Tensor, cache: _A.KVCache, block_table: torch.Tensor,
                   kv_lens: torch.Tensor, q_starts: torch.Tensor, max_q: int,
                   mask: torch.Tensor | None = None,
                   scale: float | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """``attn.tree_attention`` through ``torch.ops.w4a16.tree_attention``."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    return torch.ops.w4a16.tree_attention(q, *cache, block_table, kv_lens, q_starts, max_q, mask, scale)


@torch.library.custom_op("w4a16::token_logprobs", mutates_args=())
def _token_logprobs_op(logits: torch.Tensor, ids: torch.Tensor, top_k: int = 0
                       ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    return _S.token_logprobs(logits, ids, top_k)


@_token_logprobs_op.register_fake
def _token_logprobs_fake(logits, ids, top_k=0):
    _need(logits.dim() == 2 and logits.dtype in (*_FLOATS, torch.float32),
          "logits must be float16, bfloat16 or float32 [tokens, vocab]")
    _check_list(ids, "ids", torch.int64, logits.shape[0])
    _need(0 <= top_k <= _S.MAX_TOP and top_k <= logits.shape[1],
          f"top_k must lie in 0..{_S.MAX_TOP} and not exceed the vocabulary")
    f = [logits.new_empty(s, dtype=torch.float32) for s in (ids.shape, ids.shape, (ids.shape[0], top_k))]
    return *f, ids.new_empty((ids.shape[0], top_k))


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor, top_k: int = 0
                   ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """``scoring.token_logprobs`` through ``torch.ops.w4a16.token_logprobs``."""
    return torch.ops.w4a16.token_logprobs(logits, ids, top_k)
