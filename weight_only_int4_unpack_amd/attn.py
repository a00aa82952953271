"""Rotary positions, the paged key/value cache and attention over it.

What a decoder layer does between two weight products: the projection's output
is rotated and written into a paged cache (``kv_write``), the new tokens, plain
or drafted as a tree, attend over the cache (``tree_attention``), and the
result goes into the next product. ``rope`` rotates alone, ``kv_read`` reads
cached tokens back.

Argument marshalling only, as in ``w4a16``: shapes, types, devices and strides
are checked here, sizes and alignment again in the library, and every step of
the computation runs in its kernels. Calls enqueue on the current stream of the
tensors' device and never synchronise; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import w4a16 as _W

KV_SAME, KV_E4M3, KV_INT8 = 0, 1, 2
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}

_FORMATS = {torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
_CODES = {torch.float16: _W.F16, torch.bfloat16: _W.BF16}

# the argument structs of include/w4a16.h, in native alignment
_CACHE = "PPPPqiiii"
_ROPE = struct.Struct("@PPPPqqqqqqiiiiii")
_WRITE = struct.Struct("@" + _CACHE + "PPPPPPPqqqqqqqqqqiiii")
_ATTEND = struct.Struct("@" + _CACHE + "PPPPPPPqqqqiiiiiifi")
_READ = struct.Struct("@" + _CACHE + "PPPqii")


class KVCache(NamedTuple):
    """A paged cache: ``k`` and ``v`` ``[pages, heads, page_size, head_dim]``
    in fp16 or bf16, or, quantised, in float8_e4m3fn or int8 with fp32 scales
    ``[pages, heads, page_size]`` (value = code * scale). Slot
    ``page * page_size + offset`` holds one token."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def kv_cache(pages: int, heads: int, head_dim: int, page_size: int = 64,
             dtype: torch.dtype = torch.float8_e4m3fn, device="cuda") -> KVCache:
    """A cache of zeros."""
    shape = (pages, heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype not in _FORMATS:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.zeros(shape[:3], device=device) for _ in range(2)))


def _packed_cache(cache: KVCache, dev) -> tuple:
    """The cache's fields of an argument struct, checked."""
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("the cache's k and v must be [pages, heads, page_size, head_dim] alike")
    if v.dtype != k.dtype:
        raise ValueError("the cache's k and v must have one dtype")
    fmt = _FORMATS.get(k.dtype)
    if fmt is None:
        if k.dtype not in _CODES:
            raise ValueError("a cache holds float16, bfloat16, float8_e4m3fn or int8")
        fmt = KV_SAME
        if ks is not None or vs is not None:
            raise ValueError("a 16-bit cache has no scales")
        scales = (0, 0)
    else:
        if ks is None or vs is None:
            raise ValueError("a quantised cache needs k_scale and v_scale")
        if ks.shape != shape[:3] or vs.shape != shape[:3] or ks.dtype != torch.float32 \
                or vs.dtype != torch.float32:
            raise ValueError(f"scales must be float32 {list(shape[:3])}")
        if ks.device != dev or vs.device != dev:
            raise ValueError("all tensors must be on the same GPU")
        if not ks.is_contiguous() or not vs.is_contiguous():
            raise ValueError("the cache must be contiguous")
        scales = (ks.data_ptr(), vs.data_ptr())
    if k.device != dev or v.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    if not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("the cache must be contiguous")
    return (k.data_ptr(), v.data_ptr(), *scales, shape[0], shape[2], shape[1], shape[3], fmt)


def _heads(x: torch.Tensor, what: str):
    """Device, dtype code and (token, head) strides of an array of heads."""
    if x.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim]")
    code = _CODES.get(x.dtype)
    if code is None:
        raise ValueError(f"{what} must be float16 or bfloat16")
    if not x.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    st, sh, sd = x.stride()
    if sd != 1 and x.shape[2] != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return code, st, sh


def _array(x: torch.Tensor, what: str, dtype, dev, *shape):
    """Address of a contiguous array of the given dtype and shape."""
    if x.dtype != dtype or tuple(x.shape) != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {x.dtype} {list(x.shape)}")
    if x.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return x.data_ptr()


def _table(table: torch.Tensor, dev):
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 [positions, rot_dim]")
    if table.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    return table.data_ptr(), table.shape[0], table.shape[1]


def _out_heads(out, like: torch.Tensor, what: str):
    """The output array (made if None), and its (token, head) strides."""
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
    elif out.shape != like.shape or out.dtype != like.dtype or out.device != like.device:
        raise ValueError(f"{what} must have the input's shape, dtype and device")
    _, st, sh = _heads(out, what)
    return out, st, sh


def _call(fn, dev, *args):
    """One library call on the current stream of `dev`."""
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)   # without a Stream object: 0.1 us, not 1.9
    if index == torch._C._cuda_getDevice():              # 0.1 us, not 0.25
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _W._check(status)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original: float = 0.0, low: float = 1.0,
                     high: float = 32.0) -> list[float]:
    """The ``rot_dim / 2`` rotary frequencies, scaled for a context ``factor``
    times as long as the ``original`` one: "none", "linear", "ntk" (a larger
    base), "bands" (by the number of turns, linear between ``low`` and
    ``high``) or "ramp" (linear in the index between those)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    args = struct.pack("@dddddii", base, factor, original, low, high, rot_dim,
                       ROPE_SCALINGS[scaling])
    _W._check(_W.lib().w4a16_rope_frequencies(args, out))
    return list(out)


def rope_table(positions: int, frequencies, amplitude: float = 1.0, device="cuda") -> torch.Tensor:
    """fp32 ``[positions, rot_dim]``: each position's cosines, then its sines,
    times ``amplitude`` (angles in fp64). ``frequencies``: the ``rot_dim / 2``
    values of ``rope_frequencies``, or any others."""
    f = [float(x) for x in frequencies]
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("a table is made on a GPU")
    if positions < 0:
        raise ValueError("positions must be >= 0")
    table = torch.empty((positions, 2 * len(f)), dtype=torch.float32, device=dev)
    _call(_W.lib().w4a16_rope_table, table.device, (ctypes.c_double * max(1, len(f)))(*f),
          2 * len(f), amplitude, positions, table.data_ptr())
    return table


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
         interleaved: bool = False, inverse: bool = False,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotates the first ``table.shape[1]`` dims of every head of ``x``
    ``[tokens, heads, head_dim]`` to its token's position: halves, or
    ``interleaved`` neighbours, paired; ``inverse`` rotates back. ``x`` may be
    a view whose last dimension is contiguous; ``out=x`` rotates in place. A
    position outside the table gives NaN."""
    code, st, sh = _heads(x, "x")
    T, H, D = x.shape
    dev = x.device
    out, ot, oh = _out_heads(out, x, "out")
    pos = _array(positions, "positions", torch.int64, dev, T)
    tab, rows, rot = _table(table, dev)
    _call(_W.lib().w4a16_rope, dev,
          _ROPE.pack(x.data_ptr(), out.data_ptr(), pos, tab, T, st, sh, ot, oh, rows, H, D, rot,
                     interleaved, inverse, code))
    return out


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: KVCache,
             positions: torch.Tensor | None = None, table: torch.Tensor | None = None,
             interleaved: bool = False, q: torch.Tensor | None = None,
             q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Writes ``k`` and ``v`` ``[tokens, heads, head_dim]`` into the ``slots``
    (int64 ``[tokens]``, no two alike; a negative one is skipped) of ``cache``,
    quantised as the cache is. With ``positions`` and ``table`` ``k`` is rotated first, and
    ``q`` ``[tokens, q_heads, head_dim]``, if given, is rotated into ``q_out``
    (returned; ``q_out=q`` in place), all in one pass."""
    code, kt, kh = _heads(k, "k")
    vcode, vt, vh = _heads(v, "v")
    T, H, D = k.shape
    dev = k.device
    if v.shape != k.shape or vcode != code or v.device != dev:
        raise ValueError("k and v must have one shape, dtype and device")
    fields = _packed_cache(cache, dev)
    if fields[6] != H or fields[7] != D:
        raise ValueError(f"the cache holds {fields[6]} heads of {fields[7]} dims, k has {H} of {D}")
    if fields[8] == KV_SAME and cache.k.dtype != k.dtype:
        raise ValueError("a 16-bit cache must have k's dtype")
    at = _array(slots, "slots", torch.int64, dev, T)
    if (positions is None) != (table is None):
        raise ValueError("positions and table go together")
    pos = tab = rows = rot = 0
    if table is not None:
        pos = _array(positions, "positions", torch.int64, dev, T)
        tab, rows, rot = _table(table, dev)
    qp = op = qt = qh = ot = oh = hq = 0
    if q is not None:
        if table is None:
            raise ValueError("q is given to be rotated: positions and table are needed")
        qcode, qt, qh = _heads(q, "q")
        if qcode != code or q.device != dev or q.shape[0] != T or q.shape[2] != D:
            raise ValueError("q must be [tokens, q_heads, head_dim] like k")
        q_out, ot, oh = _out_heads(q_out, q, "q_out")
        qp, op, hq = q.data_ptr(), q_out.data_ptr(), q.shape[1]
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    _call(_W.lib().w4a16_kv_write, dev,
          _WRITE.pack(*fields, k.data_ptr(), v.data_ptr(), at, qp, op, pos, tab, T, kt, kh, vt, vh,
                      qt, qh, ot, oh, rows, hq, rot, interleaved, code))
    return q_out


def kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype | None = None,
            k_out: torch.Tensor | None = None,
            v_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Keys and values ``[tokens, heads, head_dim]`` of the given slots, in
    ``dtype`` (a 16-bit cache's own, else bfloat16 by default). A slot outside
    the cache gives zeros."""
    dev = cache.k.device
    if not cache.k.is_cuda:
        raise ValueError("all tensors must be on the same GPU")
    fields = _packed_cache(cache, dev)
    if dtype is None:
        dtype = cache.k.dtype if fields[8] == KV_SAME else torch.bfloat16
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError("dtype must be float16 or bfloat16")
    if fields[8] == KV_SAME and dtype != cache.k.dtype:
        raise ValueError("a 16-bit cache is read in its own dtype")
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D")
    T = slots.shape[0]
    at = _array(slots, "slots", torch.int64, dev, T)
    shape = (T, fields[6], fields[7])
    outs = []
    for x, what in ((k_out, "k_out"), (v_out, "v_out")):
        if x is None:
            x = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _array(x, what, dtype, dev, *shape)
        outs.append(x)
    _call(_W.lib().w4a16_kv_read, dev,
          _READ.pack(*fields, at, outs[0].data_ptr(), outs[1].data_ptr(), T, code, 0))
    return outs[0], outs[1]


def tree_attention_workspace_bytes(sequences: int, max_q: int, q_heads: int, kv_heads: int,
                                   head_dim: int, num_cus: int = 256) -> int:
    """Scratch bytes of ``tree_attention`` (host only)."""
    n = ctypes.c_int64(0)
    _W._check(_W.lib().w4a16_tree_attention_workspace_bytes(sequences, max_q, q_heads, kv_heads,
                                                            head_dim, num_cus, ctypes.byref(n)))
    return n.value


def tree_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                   kv_lens: torch.Tensor, q_starts: torch.Tensor, max_q: int,
                   mask: torch.Tensor | None = None, scale: float | None = None,
                   out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Attention of new tokens over the cache, their own keys and values
    included (``kv_write`` them first). ``q`` ``[tokens, q_heads, head_dim]``
    holds sequence b's new tokens in rows ``q_starts[b]:q_starts[b + 1]``
    (int32 ``[sequences + 1]``; at most ``max_q`` each); its ``kv_lens[b]``
    (int32) cached tokens, the new ones last, lie in the pages
    ``block_table[b]`` (int32 ``[sequences, pages]``; one row may be expanded
    to all sequences).

    New token i sees everything before the new ones and, of the new ones, j <= i
    or, with ``mask`` (int64 ``[tokens, words]``), those whose bit j % 64 of word
    j / 64 is set (``tree_mask`` makes one from parents). ``scale`` defaults to
    head_dim ** -0.5. Returns ``(out, lse)``: ``out`` like ``q`` and the natural
    log of the softmax denominator, fp32 ``[tokens, q_heads]``; 0 and -inf where
    a token sees nothing."""
    code, qt, qh = _heads(q, "q")
    T, H, D = q.shape
    dev = q.device
    fields = _packed_cache(cache, dev)
    heads, dim, fmt = fields[6:]
    if dim != D or H % heads != 0:
        raise ValueError(f"q has {H} heads of {D} dims, the cache {heads} of {dim}")
    if fmt == KV_SAME and cache.k.dtype != q.dtype:
        raise ValueError("a 16-bit cache must have q's dtype")
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.device != dev:
        raise ValueError("block_table must be int32 [sequences, pages] on q's device")
    B, pages = block_table.shape
    bs, b1 = block_table.stride()
    if b1 != 1 and pages > 1:
        raise ValueError("block_table: the last dimension must be contiguous")
    if B <= 1:
        bs = pages                          # no other row to go to
    lens = _array(kv_lens, "kv_lens", torch.int32, dev, B)
    starts = _array(q_starts, "q_starts", torch.int32, dev, B + 1)
    mp = words = 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[1] < 1:
            raise ValueError("mask must be int64 [tokens, words]")
        words = mask.shape[1]
        mp = _array(mask, "mask", torch.int64, dev, T, words)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _array(out, "out", q.dtype, dev, T, H, D)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _array(lse, "lse", torch.float32, dev, T, H)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    need = tree_attention_workspace_bytes(B, max_q, H, heads, D, _W._num_cus(dev))
    ws = _W.stream_workspace(dev, need)
    _call(_W.lib().w4a16_tree_attention, dev,
          _ATTEND.pack(*fields, q.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       block_table.data_ptr(), lens, starts, mp, T, qt, qh, bs, B, pages,
                       max_q, H, words, code, scale, 0), _W._ptr(ws), need)
    return out, lse


def tree_mask(parents: list[list[int]], device="cuda") -> torch.Tensor:
    """The mask of drafted trees: ``parents[b][j]`` is the drafted token that j
    of sequence b follows, -1 for one that follows the cached tokens. Row i has
    the bits of i and its ancestors."""
    words = max(1, max((len(p) + 63) // 64 for p in parents)) if parents else 1
    rows = []
    for tree in parents:
        seen: list[int] = []
        for j, parent in enumerate(tree):
            if not -1 <= parent < j:
                raise ValueError(f"token {j} must follow an earlier one or -1, got {parent}")
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        for m in seen:
            row = [m >> 64 * w & 2**64 - 1 for w in range(words)]
            rows.append([x - 2**64 if x >= 2**63 else x for x in row])
    return torch.tensor(rows, dtype=torch.int64, device=device).reshape(len(rows), words)
