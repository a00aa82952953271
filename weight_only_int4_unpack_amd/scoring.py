"""Log probabilities of given tokens, entropy, and the largest alternatives; verification of
drafted tokens.

Argument marshalling only, as in ``w4a16``; the computation is one pass over
the logits in the library's kernels.
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
_VERIFY = struct.Struct("@PPPPPPPPPPPqqqqiiii")
MAX_NODES = 1024                                           # of a verified sequence


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


def verify_workspace_bytes(tokens: int, vocab: int, sequences: int, max_q: int, dtype: torch.dtype,
                           num_cus: int = 256) -> int:
    """Scratch bytes of ``verify_drafts`` (host only)."""
    n = ctypes.c_int64(0)
    _W._check(_W.lib().w4a16_verify_drafts_workspace_bytes(tokens, vocab, sequences, max_q,
                                                           _CODES.get(dtype, -1), num_cus, ctypes.byref(n)))
    return n.value


def _matrix(x: torch.Tensor, what: str):
    """Row stride of a matrix whose rows may lie apart."""
    row, one = x.stride()
    if one != 1 and x.shape[1] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return row


def verify_drafts(logits: torch.Tensor, ids: torch.Tensor, q_starts: torch.Tensor, max_q: int,
                  uniforms: torch.Tensor, final_uniforms: torch.Tensor,
                  parents: torch.Tensor | None = None, draft_probs: torch.Tensor | None = None,
                  temperatures: torch.Tensor | None = None
                  ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """How far each sequence's drafted tokens are accepted, and the token after them:
    ``(tokens, path, counts)``, int64 and int32 ``[sequences, max_q]`` and int32
    ``[sequences]``. The first ``counts[b]`` entries of ``tokens[b]`` are the accepted tokens and one drawn after
    them; those of ``path[b]`` node 0 and the accepted nodes (``paging.kv_compact`` keeps them). The rest is -1.

    ``logits`` ``[tokens, vocab]`` (fp16, bf16 or fp32; rows may lie apart) and
    ``ids`` (int64 ``[tokens]``) have sequence b's nodes in rows
    ``q_starts[b]:q_starts[b + 1]`` (int32 ``[sequences + 1]``; at most ``max_q``,
    up to 1024, each) as ``tree_attention`` does: node 0 is the token chosen last, the others
    are drafted. ``parents`` (int32 ``[tokens]``) says which node of its sequence each follows; without
    them, the one before. ``uniforms`` (``[tokens]``) and ``final_uniforms``
    (``[sequences]``) are fp32 random numbers in [0, 1).

    Drafted tokens are taken as given (a node is accepted with the probability that the model has for its token,
    after the siblings rejected before it), or, with ``draft_probs`` (fp32
    ``[tokens, vocab]``, chains only; row i is what the token after token i was drawn
    from), by the ratio of the model's probability to the draft's, with the last token drawn from what the model
    has above the draft. Either way tokens are distributed as the model's own.
    ``temperatures``: fp32 ``[sequences]``, 1 by default; 0 is greedy. A
    row without a softmax (NaN, +inf, or all -inf) ends its sequence with -1."""
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, vocab]")
    code = _CODES.get(logits.dtype)
    if code is None:
        raise ValueError("logits must be float16, bfloat16 or float32")
    if not logits.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    T, V = logits.shape
    dev = logits.device
    row = _matrix(logits, "logits")
    if q_starts.dim() != 1 or q_starts.shape[0] < 1:
        raise ValueError("q_starts must be int32 [sequences + 1]")
    B = q_starts.shape[0] - 1
    at = _array(ids, "ids", torch.int64, dev, T)
    starts = _array(q_starts, "q_starts", torch.int32, dev, B + 1)
    u = _array(uniforms, "uniforms", torch.float32, dev, T)
    final = _array(final_uniforms, "final_uniforms", torch.float32, dev, B)
    tree = probs = stride = temps = 0
    if parents is not None:
        if draft_probs is not None:
            raise ValueError("draft_probs go with chains: parents must be None")
        tree = _array(parents, "parents", torch.int32, dev, T)
    if draft_probs is not None:
        if draft_probs.shape != logits.shape or draft_probs.dtype != torch.float32 or draft_probs.device != dev:
            raise ValueError("draft_probs must be float32 like logits, on their device")
        probs, stride = draft_probs.data_ptr(), _matrix(draft_probs, "draft_probs")
    if temperatures is not None:
        temps = _array(temperatures, "temperatures", torch.float32, dev, B)
    need = verify_workspace_bytes(T, V, B, max_q, logits.dtype, _W._num_cus(dev))
    tokens = ids.new_empty((B, max_q))
    path = q_starts.new_empty((B, max_q))
    counts = q_starts.new_empty((B,))
    ws = _W.stream_workspace(dev, need)
    _call(_W.lib().w4a16_verify_drafts, dev,
          _VERIFY.pack(logits.data_ptr(), at, starts, tree, probs, temps, u, final, tokens.data_ptr(),
                       path.data_ptr(), counts.data_ptr(), T, row, stride, V, B, max_q, code, 0),
          _W._ptr(ws), need)
    return tokens, path, counts
