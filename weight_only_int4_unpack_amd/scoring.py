"""Log probabilities of given tokens, entropy, and the largest alternatives.

Argument marshalling only, as in ``w4a16``; the computation is one pass over
the logits in the library's kernel.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import w4a16 as _W
from .attn import _array, _call

MAX_TOP = 64
F32 = 2                                                    # W4A16_F32
_CODES = {torch.float16: _W.F16, torch.bfloat16: _W.BF16, torch.float32: F32}
_ARGS = struct.Struct("@PPPPPPqqqii")


def workspace_bytes(tokens: int, vocab: int, top_k: int, num_cus: int = 256) -> int:
    """Scratch bytes of ``token_logprobs`` (host only)."""
    n = ctypes.c_int64(0)
    _W._check(_W.lib().w4a16_token_logprobs_workspace_bytes(tokens, vocab, top_k, num_cus,
                                                            ctypes.byref(n)))
    return n.value


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor, top_k: int = 0):
    """``(logprobs, entropy, top_logprobs, top_ids)`` of ``logits`` ``[tokens,
    vocab]`` (fp16, bf16 or fp32; rows may lie apart): the log probability of
    ``ids`` (int64 ``[tokens]``) and the entropy, fp32 ``[tokens]``, and the
    ``top_k`` (0 to 64) likeliest tokens' log probabilities and ids ``[tokens,
    top_k]``, descending, equal ones by lowest id. An id outside the vocabulary
    gives NaN, and so does a row without a softmax (NaN, +inf, or all -inf)."""
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, vocab]")
    code = _CODES.get(logits.dtype)
    if code is None:
        raise ValueError("logits must be float16, bfloat16 or float32")
    if not logits.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    T, V = logits.shape
    row, one = logits.stride()
    if one != 1 and V != 1:
        raise ValueError("logits: the last dimension must be contiguous")
    dev = logits.device
    at = _array(ids, "ids", torch.int64, dev, T)
    need = workspace_bytes(T, V, top_k, _W._num_cus(dev))
    logprobs = torch.empty_like(ids, dtype=torch.float32)
    entropy = torch.empty_like(logprobs)
    top = logprobs.new_empty((T, top_k))
    top_ids = ids.new_empty((T, top_k))
    ws = _W.stream_workspace(dev, need)
    _call(_W.lib().w4a16_token_logprobs, dev,
          _ARGS.pack(logits.data_ptr(), at, logprobs.data_ptr(), entropy.data_ptr(),
                     top.data_ptr(), top_ids.data_ptr(), T, row, V, top_k, code),
          _W._ptr(ws), need)
    return logprobs, entropy, top, top_ids
