"""CPU tests of the C ABI of the operators around the weight products: struct
layouts, argument checks, scratch sizes, rotary frequencies. Nothing here
launches a kernel: every call is host-only or fails its checks first."""
import ctypes
import math
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

from weight_only_int4_unpack_amd import attn, scoring
from weight_only_int4_unpack_amd import w4a16 as W

P = 0x10000                       # aligned, never dereferenced on the host
HAS_GPU = torch.cuda.is_available()
NO_DEVICE = W.OK if HAS_GPU else W.ERR_DEVICE


def _cache(**kw):
    f = dict(k=P, v=P, ks=P, vs=P, pages=4, page=64, heads=8, dim=128, fmt=attn.KV_E4M3)
    f.update(kw)
    return [f[n] for n in ("k", "v", "ks", "vs", "pages", "page", "heads", "dim", "fmt")]


def _rope(**kw):
    f = dict(x=P, out=2 * P, pos=P, table=P, T=4, xt=1024, xh=128, ot=1024, oh=128, rows=32, H=8, D=128,
             rot=128, inter=0, inverse=0, dt=1)
    f.update(kw)
    return W.lib().w4a16_rope(attn._ROPE.pack(*f.values()), None)


def _write(cache=None, **kw):
    f = dict(k=P, v=P, slots=P, q=P, qo=2 * P, pos=P, table=P, T=4, kt=1024, kh=128, vt=1024, vh=128,
             qt=1024, qh=128, ot=1024, oh=128, rows=32, hq=8, rot=128, inter=0, dt=1)
    f.update(kw)
    return W.lib().w4a16_kv_write(attn._WRITE.pack(*(cache or _cache()), *f.values()), None)


def _read(cache=None, **kw):
    f = dict(slots=P, k=P, v=P, T=4, dt=1, r=0)
    f.update(kw)
    return W.lib().w4a16_kv_read(attn._READ.pack(*(cache or _cache()), *f.values()), None)


def _attend(cache=None, ws=P, nb=1 << 40, **kw):
    f = dict(q=P, out=P, lse=P, table=P, lens=P, starts=P, mask=0, T=4, qt=1024, qh=128, stride=8,
             B=2, pages=8, max_q=2, hq=32, words=0, dt=1, scale=0.1, r=0)
    f.update(kw)
    return W.lib().w4a16_tree_attention(attn._ATTEND.pack(*(cache or _cache()), *f.values()),
                                        ws, nb, None)


def _score(ws=P, nb=1 << 40, **kw):
    f = dict(x=P, ids=P, lp=P, ent=P, top=P, top_ids=P, T=4, row=32000, V=32000, k=5, dt=1)
    f.update(kw)
    return W.lib().w4a16_token_logprobs(scoring._ARGS.pack(*f.values()), ws, nb, None)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    names = ["rope", "kv_write", "kv_read", "tree_attention", "token_logprobs", "rope_scale"]
    src.write_text('#include <stdio.h>\n#include "w4a16.h"\nint main(void) { printf("' +
                   "%zu " * len(names) + '\\n", ' +
                   ", ".join(f"sizeof(w4a16_{n}_t)" for n in names) + "); return 0; }\n")
    exe = str(tmp_path / "sizes")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    subprocess.run(["gcc", "-I", os.path.dirname(W.HEADER), str(src), "-o", exe], check=True, env=env)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, env=env).stdout
    want = [attn._ROPE.size, attn._WRITE.size, attn._READ.size, attn._ATTEND.size,
            scoring._ARGS.size, struct.calcsize("@dddddii")]
    assert [int(x) for x in out.split()] == want


CACHE_REFUSALS = [
    (dict(fmt=3), W.ERR_DTYPE), (dict(dim=120), W.ERR_SHAPE), (dict(dim=0), W.ERR_SHAPE),
    (dict(dim=264), W.ERR_SHAPE), (dict(dim=136, fmt=0), W.ERR_SHAPE), (dict(page=48), W.ERR_SHAPE),
    (dict(page=8), W.ERR_SHAPE), (dict(page=8192), W.ERR_SHAPE), (dict(heads=0), W.ERR_SHAPE),
    (dict(pages=-1), W.ERR_SHAPE), (dict(k=0), W.ERR_NULL), (dict(ks=0), W.ERR_NULL),
    (dict(v=P + 8), W.ERR_ALIGN), (dict(vs=P + 4), W.ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(kw, status):
    cache = _cache(**kw)
    assert _write(cache) == status and W.last_error()
    assert _read(cache) == status
    assert _attend(cache) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), W.ERR_DTYPE), (dict(D=12), W.ERR_SHAPE), (dict(T=-1), W.ERR_SHAPE),
    (dict(T=1 << 30), W.ERR_SHAPE), (dict(H=-1), W.ERR_SHAPE), (dict(rot=3), W.ERR_SHAPE),
    (dict(rot=130), W.ERR_SHAPE), (dict(rot=0), W.ERR_SHAPE), (dict(rows=0), W.ERR_SHAPE),
    (dict(x=0), W.ERR_NULL), (dict(pos=0), W.ERR_NULL), (dict(table=0), W.ERR_NULL),
    (dict(x=P + 2), W.ERR_ALIGN), (dict(xt=1025), W.ERR_ALIGN), (dict(oh=4), W.ERR_ALIGN),
    (dict(xh=-128), W.ERR_SHAPE), (dict(out=P, ot=2048), W.ERR_SHAPE), (dict(table=P + 4), W.ERR_ALIGN),
    (dict(T=0, x=0), W.OK), (dict(H=0, x=0), W.OK),
])
def test_rope_refusals(kw, status):
    assert _rope(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), W.ERR_DTYPE), (dict(k=0), W.ERR_NULL), (dict(slots=0), W.ERR_NULL),
    (dict(qo=0), W.ERR_NULL), (dict(pos=0), W.ERR_NULL), (dict(table=0), W.ERR_NULL),
    (dict(pos=0, table=0), W.ERR_NULL),               # q without a rotation
    (dict(T=-1), W.ERR_SHAPE), (dict(hq=-1), W.ERR_SHAPE), (dict(rot=129), W.ERR_SHAPE),
    (dict(vt=12), W.ERR_ALIGN), (dict(v=P + 8), W.ERR_ALIGN), (dict(qh=1 << 40), W.ERR_SHAPE),
    (dict(qo=P, ot=8), W.ERR_SHAPE), (dict(T=0, k=0), W.OK),
])
def test_kv_write_refusals(kw, status):
    assert _write(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), W.ERR_DTYPE), (dict(slots=0), W.ERR_NULL), (dict(v=0), W.ERR_NULL),
    (dict(k=P + 8), W.ERR_ALIGN), (dict(T=1 << 28), W.ERR_SHAPE), (dict(T=0, k=0), W.OK),
])
def test_kv_read_refusals(kw, status):
    assert _read(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), W.ERR_DTYPE), (dict(hq=30), W.ERR_SHAPE), (dict(hq=0), W.ERR_SHAPE),
    (dict(B=-1), W.ERR_SHAPE), (dict(max_q=-1), W.ERR_SHAPE), (dict(pages=-1), W.ERR_SHAPE),
    (dict(stride=7), W.ERR_SHAPE), (dict(q=0), W.ERR_NULL), (dict(lse=0), W.ERR_NULL),
    (dict(table=0), W.ERR_NULL), (dict(lens=0), W.ERR_NULL), (dict(mask=P, words=0), W.ERR_SHAPE),
    (dict(mask=P + 4, words=1), W.ERR_ALIGN), (dict(qt=100), W.ERR_ALIGN), (dict(out=P + 8), W.ERR_ALIGN),
    (dict(scale=math.inf), W.ERR_VALUE), (dict(scale=math.nan), W.ERR_VALUE),
    (dict(max_q=1 << 30, B=1 << 19), W.ERR_SHAPE), (dict(nb=65536), W.ERR_WORKSPACE),
    (dict(ws=0), W.ERR_NULL), (dict(ws=P + 8), W.ERR_ALIGN), (dict(T=0, q=0), W.OK),
    (dict(B=0, table=0), W.OK),
])
def test_attention_refusals(kw, status):
    assert _attend(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), W.ERR_DTYPE), (dict(V=0), W.ERR_SHAPE), (dict(T=-1), W.ERR_SHAPE),
    (dict(k=65), W.ERR_SHAPE), (dict(k=-1), W.ERR_SHAPE), (dict(V=3, k=4), W.ERR_SHAPE),
    (dict(row=-1), W.ERR_SHAPE), (dict(x=0), W.ERR_NULL), (dict(top=0), W.ERR_NULL),
    (dict(x=P + 1), W.ERR_ALIGN), (dict(x=P + 2, dt=2), W.ERR_ALIGN), (dict(ids=P + 4), W.ERR_ALIGN),
    (dict(nb=65536), W.ERR_WORKSPACE), (dict(ws=0), W.ERR_NULL), (dict(T=0, x=0), W.OK),
])
def test_token_logprobs_refusals(kw, status):
    assert _score(**kw) == status


def test_null_arguments():
    L = W.lib()
    for f in (L.w4a16_rope, L.w4a16_kv_write, L.w4a16_kv_read):
        assert f(None, None) == W.ERR_NULL
    assert L.w4a16_tree_attention(None, None, 0, None) == W.ERR_NULL
    assert L.w4a16_token_logprobs(None, None, 0, None) == W.ERR_NULL
    assert L.w4a16_rope_frequencies(None, None) == W.ERR_NULL
    assert L.w4a16_rope_table(None, 128, 1.0, 4, P, None) == W.ERR_NULL
    assert L.w4a16_rope_table((ctypes.c_double * 64)(), 127, 1.0, 4, P, None) == W.ERR_SHAPE
    assert L.w4a16_rope_table((ctypes.c_double * 64)(), 128, 1.0, 0, None, None) == W.OK


@pytest.mark.skipif(HAS_GPU, reason="would launch")
def test_good_arguments_reach_the_device_check():
    assert _rope() == _write() == _read() == _attend() == _score() == W.ERR_DEVICE


def test_workspace_sizes():
    # attention: the counters and a part for each item; none once rows fill the device alone
    small = attn.tree_attention_workspace_bytes(1, 1, 32, 8, 128)
    assert small > W.WORKSPACE_COUNTER_BYTES and small % 4 == 0
    assert attn.tree_attention_workspace_bytes(64, 4096, 32, 8, 128) == 0
    for B, n, H, Hk, D in [(1, 1, 1, 1, 8), (64, 1, 40, 8, 128), (3, 77, 14, 2, 80), (300, 2, 8, 8, 256)]:
        assert 0 <= attn.tree_attention_workspace_bytes(B, n, H, Hk, D) < 1 << 28
    # scores: one part per split, at most 64, none for a row of one tile
    assert scoring.workspace_bytes(1, 8192, 20) == 0
    assert scoring.workspace_bytes(1, 8193, 20) == W.WORKSPACE_COUNTER_BYTES + 2 * (16 + 160)
    assert scoring.workspace_bytes(5000, 151936, 20) == 0
    with pytest.raises(W.W4A16Error):
        scoring.workspace_bytes(1, 0, 0)


# ---------------------------------------------------------------- frequencies
def _plain(r, base):
    return [base ** (-2.0 * i / r) for i in range(r // 2)]


@pytest.mark.parametrize("r", [2, 20, 64, 128, 256])
def test_frequencies_unscaled_linear_ntk(r):
    f = _plain(r, 5e5)
    assert np.allclose(attn.rope_frequencies(r, 5e5), f, rtol=1e-14)
    assert np.allclose(attn.rope_frequencies(r, 5e5, "linear", 8.0), [x / 8 for x in f], rtol=1e-14)
    if r > 2:
        got = attn.rope_frequencies(r, 5e5, "ntk", 8.0)
        assert np.allclose(got, _plain(r, 5e5 * 8.0 ** (r / (r - 2))), rtol=1e-13)
        # the slowest frequency is scaled by the factor, the fastest not at all
        assert math.isclose(got[-1], f[-1] / 8, rel_tol=1e-12) and got[0] == 1.0


def test_frequencies_by_bands():
    r, base, s, original, low, high = 128, 5e5, 8.0, 8192.0, 1.0, 4.0
    got = attn.rope_frequencies(r, base, "bands", s, original, low, high)
    seen = set()
    for f, g in zip(_plain(r, base), got):
        turns = original * f / (2 * math.pi)
        if turns >= high:
            seen.add("kept"); want = f
        elif turns <= low:
            seen.add("scaled"); want = f / s
        else:
            seen.add("between")
            a = (turns - low) / (high - low)
            want = a * f + (1 - a) * f / s
        assert math.isclose(g, want, rel_tol=1e-12)
    assert seen == {"kept", "scaled", "between"}


def test_frequencies_by_ramp():
    r, base, s, original, low, high = 128, 1e4, 4.0, 4096.0, 1.0, 32.0
    got = attn.rope_frequencies(r, base, "ramp", s, original, low, high)
    f = _plain(r, base)
    index = lambda n: r * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    i0, i1 = math.floor(index(high)), math.ceil(index(low))
    assert 0 < i0 < i1 < r // 2
    for i in range(r // 2):
        a = min(max((i - i0) / (i1 - i0), 0.0), 1.0)
        assert math.isclose(got[i], (1 - a) * f[i] + a * f[i] / s, rel_tol=1e-12)


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=3), W.ERR_SHAPE), (dict(rot_dim=258), W.ERR_SHAPE), (dict(base=1.0), W.ERR_VALUE),
    (dict(base=math.nan), W.ERR_VALUE), (dict(scaling="linear", factor=0.5), W.ERR_VALUE),
    (dict(scaling="ntk", factor=2.0, rot_dim=2), W.ERR_SHAPE),
    (dict(scaling="bands", factor=2.0), W.ERR_VALUE),                       # original is 0
    (dict(scaling="ramp", factor=2.0, original=4096.0, low=4.0, high=1.0), W.ERR_VALUE),
])
def test_frequency_refusals(kw, status):
    with pytest.raises(W.W4A16Error) as e:
        attn.rope_frequencies(**{"rot_dim": 128, **kw})
    assert e.value.status == status


def test_unknown_scaling_and_cpu_tensors():
    with pytest.raises(ValueError):
        attn.rope_frequencies(128, scaling="other")
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    pos, table = torch.zeros(2, dtype=torch.int64), torch.zeros((8, 64))
    with pytest.raises(ValueError):
        attn.rope(x, pos, table)
    with pytest.raises(ValueError):
        attn.kv_read(attn.KVCache(*[torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)] * 2), pos)
    with pytest.raises(ValueError):
        scoring.token_logprobs(torch.zeros((2, 9)), pos)


def test_tree_mask_rows():
    m = attn.tree_mask([[-1, 0, 0, 2], [-1]], device="cpu")
    assert m.tolist() == [[0b0001], [0b0011], [0b0101], [0b1101], [0b1]]
    chain = attn.tree_mask([list(range(-1, 69))], device="cpu")
    assert chain.shape == (70, 2) and chain[69].tolist() == [-1, 63]
    with pytest.raises(ValueError):
        attn.tree_mask([[0]], device="cpu")
