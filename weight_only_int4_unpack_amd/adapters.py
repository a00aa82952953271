"""Low-rank adapters of many requests beside a product that all share.

``lora`` adds to each token's row of a product (``w4a16.gemm``'s) what its
request's adapter makes of the same input; ``lora_plan`` orders a step's tokens
by adapter once for all products of the step.

Argument marshalling only, as in ``w4a16``: shapes, types, devices and strides
are checked here, sizes and alignment again in the library. Calls enqueue on the
current stream of the tensors' device and never synchronise; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple

import torch

from . import w4a16 as _W
from .attn import _CODES, _array, _call

MAX_ADAPTERS = 1024
MAX_RANK = 128
_ARGS = struct.Struct("@PPPPPPPPqqqqiiiiii")


class LoraPlan(NamedTuple):
    """Which adapter each token of a step takes, as ``lora`` reads it."""
    data: torch.Tensor
    tokens: int
    adapters: int


@functools.lru_cache(maxsize=4096)
def plan_bytes(tokens: int, adapters: int) -> int:
    """Bytes of a plan (host only)."""
    n = ctypes.c_int64(0)
    _W._check(_W.lib().w4a16_lora_plan_bytes(tokens, adapters, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=4096)
def workspace_bytes(tokens: int, k: int, n: int, adapters: int, rank: int, num_cus: int = 256) -> int:
    """Scratch bytes of ``lora`` (host only)."""
    need = ctypes.c_int64(0)
    _W._check(_W.lib().w4a16_lora_workspace_bytes(tokens, k, n, adapters, rank, num_cus, ctypes.byref(need)))
    return need.value


def lora_plan(index: torch.Tensor, adapters: int, nbytes: int = 0) -> LoraPlan:
    """The plan of a step whose token t takes adapter ``index[t]`` (int32
    ``[tokens]``) of ``adapters`` (1 to 1024); anything outside, such as -1: none.
    Its memory has ``plan_bytes``, or ``nbytes`` if that is more."""
    if index.dim() != 1:
        raise ValueError("index must be int32 [tokens]")
    if not index.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    T, dev = index.shape[0], index.device
    at = _array(index, "index", torch.int32, dev, T)
    data = index.new_empty(max(plan_bytes(T, adapters), nbytes), dtype=torch.uint8)
    _call(_W.lib().w4a16_lora_plan, dev, at, T, adapters, data.data_ptr())
    return LoraPlan(data, T, adapters)


def _rows(x: torch.Tensor, what: str, code, dev, *shape):
    """Address and row stride of a 16-bit matrix."""
    if tuple(x.shape) != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(x.shape)}")
    if _CODES.get(x.dtype) != code:
        raise ValueError(f"{what} must have x's dtype")
    if x.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    row, one = x.stride()
    if one != 1 and shape[1] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return x.data_ptr(), row if shape[0] > 1 else shape[1]


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, plan: LoraPlan,
         base: torch.Tensor | None = None, scales: torch.Tensor | None = None,
         ranks: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """``base[t] + scales[i] * (x[t] @ a[i].T) @ b[i].T`` for each token t and its
    adapter i by ``plan``; ``base[t]`` where it has none.

    ``x`` ``[tokens, k]`` fp16 or bf16, ``a`` ``[adapters, rank, k]`` and ``b``
    ``[adapters, n, rank]`` in its dtype (rank a multiple of 8, up to 128);
    ``base`` ``[tokens, n]``, zeros by default; ``scales`` fp32 ``[adapters]``, 1 by
    default; ``ranks`` int32 ``[adapters]``: what lies from an adapter's own rank on
    takes no part. Rows of ``x``, ``base`` and ``out`` may lie apart; ``out=base``
    adds in place, any other ``out`` is apart from all that is read. fp32 sums, one rounding."""
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x must be [tokens, k], a [adapters, rank, k], b [adapters, n, rank]")
    code = _CODES.get(x.dtype)
    if code is None:
        raise ValueError("x must be float16 or bfloat16")
    if not x.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    T, K = x.shape
    R, rank, _ = a.shape
    N = b.shape[1]
    dev = x.device
    xp, xs = _rows(x, "x", code, dev, T, K)
    ap = _array(a, "a", x.dtype, dev, R, rank, K)
    bp = _array(b, "b", x.dtype, dev, R, N, rank)
    if plan.tokens != T or plan.adapters != R:
        raise ValueError(f"the plan is for {plan.tokens} tokens and {plan.adapters} adapters, not {T} and {R}")
    data = plan.data
    if data.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    if data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() < plan_bytes(T, R):
        raise ValueError("plan.data must be lora_plan's")
    basep = bs = 0
    if base is not None:
        basep, bs = _rows(base, "base", code, dev, T, N)
    if out is None:
        # like `base` where that is as it should be: 0.9 us, not 1.5
        out = torch.empty_like(base) if base is not None and base.is_contiguous() else x.new_empty((T, N))
        outp, os = out.data_ptr(), N
    else:
        outp, os = _rows(out, "out", code, dev, T, N)
    sp = 0 if scales is None else _array(scales, "scales", torch.float32, dev, R)
    rp = 0 if ranks is None else _array(ranks, "ranks", torch.int32, dev, R)
    need = workspace_bytes(T, K, N, R, rank, _W._num_cus(dev))
    ws = _W.stream_workspace(dev, need)
    _call(_W.lib().w4a16_lora, dev,
          _ARGS.pack(xp, ap, bp, basep, outp, sp, rp, data.data_ptr(), T, xs, bs, os, K, N, R, rank,
                     code, 0), _W._ptr(ws), need)
    return out
