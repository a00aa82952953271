"""CPU tests of the C ABI of the operators of a batch of requests (verification of drafts,
pages of the cache, adapters): struct layouts, argument checks, scratch sizes. Nothing here
launches a kernel: every call is host-only or fails its checks first."""
import ctypes
import os
import shutil
import struct
import subprocess

import pytest
import torch

from weight_only_int4_unpack_amd import adapters, attn, paging, scoring
from weight_only_int4_unpack_amd import w4a16 as W

P = 0x10000                       # aligned, never dereferenced on the host
HAS_GPU = torch.cuda.is_available()
NO_DEVICE = W.OK if HAS_GPU else W.ERR_DEVICE


def _verify(ws=P, nb=1 << 40, **kw):
    f = dict(x=P, ids=P, starts=P, parents=0, probs=P, temps=P, u=P, final=P, tokens=P, path=P, counts=P,
             T=8, row=32000, prow=32000, V=32000, B=2, max_q=4, dt=1, r=0)
    f.update(kw)
    return W.lib().w4a16_verify_drafts(scoring._VERIFY.pack(*f.values()), ws, nb, None)


def _pages(fork=False, **kw):
    f = dict(refs=P, table=P, lens=P, pages=64, stride=8, rows=4, entries=8, page=16, r=0, a=P, b=P, served=P, src=P,
             dst=P, n=3, r2=0)
    f.update(kw)
    fn = W.lib().w4a16_pages_fork if fork else W.lib().w4a16_pages_resize
    return fn(paging._PAGES.pack(*f.values()), None)


def _cache(**kw):
    f = dict(k=P, v=P, ks=P, vs=P, pages=4, page=64, heads=8, dim=128, fmt=attn.KV_E4M3)
    f.update(kw)
    return list(f.values())


def _held(*caches):
    data = b"".join(paging._FIELDS.pack(*c) for c in caches)
    return (ctypes.c_char * len(data)).from_buffer_copy(data)


def _copy(group=None, **kw):
    held = _held(*(group or [_cache(), _cache()]))
    f = dict(caches=ctypes.addressof(held), src=P, dst=P, n=2, count=len(group or [0, 0]), r=0)
    f.update(kw)
    return W.lib().w4a16_kv_copy_pages(paging._COPY.pack(*f.values()), None)


def _compact(group=None, **kw):
    held = _held(*(group or [_cache(), _cache()]))
    f = dict(caches=ctypes.addressof(held), table=P, lens=P, starts=P, path=P, counts=P, new=2 * P, stride=8, B=2,
             entries=8, width=4, count=len(group or [0, 0]))
    f.update(kw)
    return W.lib().w4a16_kv_compact(paging._COMPACT.pack(*f.values()), None)


def _lora(ws=P, nb=1 << 40, **kw):
    f = dict(x=2 * P, a=P, b=P, base=P, out=P, scales=P, ranks=P, plan=P, T=4, xs=16384, bs=1024, os=1024, k=16384, n=1024,
             R=4, rank=16, dt=1, r=0)
    f.update(kw)
    return W.lib().w4a16_lora(adapters._ARGS.pack(*f.values()), ws, nb, None)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    names = ["verify_drafts", "pages", "page_pool", "kv_copy_pages", "kv_compact", "lora", "kv_cache"]
    src.write_text('#include <stdio.h>\n#include "w4a16.h"\nint main(void) { printf("' +
                   "%zu " * len(names) + '\\n", ' +
                   ", ".join(f"sizeof(w4a16_{n}_t)" for n in names) + "); return 0; }\n")
    exe = str(tmp_path / "sizes")
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    subprocess.run(["gcc", "-I", os.path.dirname(W.HEADER), str(src), "-o", exe], check=True, env=env)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, env=env).stdout
    want = [scoring._VERIFY.size, paging._PAGES.size, struct.calcsize("@PPPqqiiii"), paging._COPY.size,
            paging._COMPACT.size, adapters._ARGS.size, paging._FIELDS.size]
    assert [int(x) for x in out.split()] == want


def test_good_arguments_reach_the_device_check():
    if HAS_GPU:
        pytest.skip("the addresses are not real")
    assert [_verify(), _verify(parents=P, probs=0), _pages(), _pages(True), _copy(), _compact(), _lora()] == \
        [W.ERR_DEVICE] * 7
    assert W.lib().w4a16_lora_plan(P, 4, 4, P, None) == W.ERR_DEVICE


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), W.ERR_DTYPE), (dict(V=0), W.ERR_SHAPE), (dict(V=(1 << 20) + 1), W.ERR_SHAPE),
    (dict(T=-1), W.ERR_SHAPE), (dict(T=1 << 40), W.ERR_SHAPE), (dict(B=-1), W.ERR_SHAPE),
    (dict(B=(1 << 20) + 1), W.ERR_SHAPE), (dict(max_q=-1), W.ERR_SHAPE), (dict(max_q=1025), W.ERR_SHAPE),
    (dict(parents=P), W.ERR_SHAPE),                   # draft_probs go with chains
    (dict(row=-1), W.ERR_SHAPE), (dict(prow=1 << 40), W.ERR_SHAPE), (dict(x=0), W.ERR_NULL),
    (dict(ids=0), W.ERR_NULL), (dict(starts=0), W.ERR_NULL), (dict(u=0), W.ERR_NULL), (dict(final=0), W.ERR_NULL),
    (dict(tokens=0), W.ERR_NULL), (dict(path=0), W.ERR_NULL), (dict(counts=0), W.ERR_NULL),
    (dict(x=P + 1), W.ERR_ALIGN), (dict(x=P + 2, dt=2), W.ERR_ALIGN), (dict(probs=P + 2), W.ERR_ALIGN),
    (dict(tokens=P + 4), W.ERR_ALIGN), (dict(nb=0), W.ERR_WORKSPACE), (dict(ws=0), W.ERR_NULL),
    (dict(ws=P + 8), W.ERR_ALIGN), (dict(B=0, starts=0), W.OK),
])
def test_verify_refusals(kw, status):
    assert _verify(**kw) == status
    assert status == W.OK or W.last_error()


@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(page=8), W.ERR_SHAPE), (dict(page=48), W.ERR_SHAPE), (dict(page=8192), W.ERR_SHAPE),
    (dict(pages=-1), W.ERR_SHAPE), (dict(pages=(1 << 30) + 1), W.ERR_SHAPE), (dict(rows=-1), W.ERR_SHAPE),
    (dict(entries=-1), W.ERR_SHAPE), (dict(stride=7), W.ERR_SHAPE), (dict(stride=1 << 40), W.ERR_SHAPE),
    (dict(entries=1 << 27, stride=1 << 27), W.ERR_SHAPE), (dict(n=-1), W.ERR_SHAPE), (dict(n=4097), W.ERR_SHAPE),
    (dict(refs=0), W.ERR_NULL), (dict(table=0), W.ERR_NULL), (dict(lens=0), W.ERR_NULL), (dict(a=0), W.ERR_NULL),
    (dict(b=0), W.ERR_NULL), (dict(served=0), W.ERR_NULL), (dict(src=0), W.ERR_NULL), (dict(dst=0), W.ERR_NULL),
    (dict(lens=P + 2), W.ERR_ALIGN), (dict(dst=P + 1), W.ERR_ALIGN), (dict(n=0, refs=0, a=0), W.OK),
])
def test_pages_refusals(fork, kw, status):
    assert _pages(fork, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), W.ERR_SHAPE), (dict(n=1 << 31), W.ERR_SHAPE), (dict(n=1 << 30), W.ERR_SHAPE),
    (dict(src=0), W.ERR_NULL), (dict(dst=P + 2), W.ERR_ALIGN), (dict(count=-1), W.ERR_SHAPE),
    (dict(count=4097), W.ERR_SHAPE), (dict(caches=0), W.ERR_NULL), (dict(n=0, src=0), W.OK), (dict(count=0), W.OK),
])
def test_copy_refusals(kw, status):
    assert _copy(**kw) == status


@pytest.mark.parametrize("other", [dict(pages=5), dict(page=32), dict(heads=4), dict(dim=64), dict(fmt=attn.KV_INT8)])
def test_caches_of_a_group_are_alike(other):
    pair = [_cache(), _cache(**other)]
    assert _copy(pair) == W.ERR_SHAPE and "cache 1" in W.last_error()
    assert _compact(pair) == W.ERR_SHAPE


@pytest.mark.parametrize("bad,status", [(dict(k=0), W.ERR_NULL), (dict(vs=0), W.ERR_NULL), (dict(page=8), W.ERR_SHAPE),
                                        (dict(dim=120), W.ERR_SHAPE), (dict(v=P + 8), W.ERR_ALIGN)])
def test_every_cache_of_a_group_is_checked(bad, status):
    assert _copy([_cache(), _cache(**bad)]) == status
    assert _compact([_cache(), _cache(**bad)]) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), W.ERR_SHAPE), (dict(B=(1 << 20) + 1), W.ERR_SHAPE), (dict(width=-1), W.ERR_SHAPE),
    (dict(entries=-1), W.ERR_SHAPE), (dict(stride=7), W.ERR_SHAPE), (dict(stride=0), W.ERR_SHAPE),
    (dict(new=P), W.ERR_SHAPE),                       # in place of kv_lens
    (dict(lens=0), W.ERR_NULL), (dict(path=0), W.ERR_NULL), (dict(counts=0), W.ERR_NULL), (dict(new=0), W.ERR_NULL),
    (dict(table=0), W.ERR_NULL), (dict(path=P + 2), W.ERR_ALIGN), (dict(B=0, lens=0), W.OK),
])
def test_compact_refusals(kw, status):
    assert _compact(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), W.ERR_DTYPE), (dict(T=-1), W.ERR_SHAPE), (dict(T=(1 << 24) + 1), W.ERR_SHAPE),
    (dict(R=0), W.ERR_SHAPE), (dict(R=1025), W.ERR_SHAPE), (dict(rank=0), W.ERR_SHAPE), (dict(rank=12), W.ERR_SHAPE),
    (dict(rank=136), W.ERR_SHAPE), (dict(k=12), W.ERR_SHAPE), (dict(k=0), W.ERR_SHAPE), (dict(n=4), W.ERR_SHAPE),
    (dict(n=1 << 23), W.ERR_SHAPE), (dict(xs=513), W.ERR_ALIGN), (dict(os=1016), W.ERR_SHAPE), (dict(xs=-8), W.ERR_SHAPE),
    (dict(bs=1 << 40), W.ERR_SHAPE), (dict(x=0), W.ERR_NULL), (dict(a=0), W.ERR_NULL), (dict(b=0), W.ERR_NULL),
    (dict(out=0), W.ERR_NULL), (dict(plan=0), W.ERR_NULL), (dict(x=P + 2), W.ERR_ALIGN), (dict(plan=P + 8), W.ERR_ALIGN),
    (dict(scales=P + 2), W.ERR_ALIGN), (dict(bs=2048), W.ERR_SHAPE),   # base is out, at another stride
    (dict(x=P), W.ERR_SHAPE),                         # out would be read as x
    (dict(nb=0), W.ERR_WORKSPACE), (dict(ws=0), W.ERR_NULL), (dict(T=0, x=0), W.OK),
    (dict(nb=0, ws=0, xs=512, k=512), W.ERR_DEVICE),  # one kernel does both
])
def test_lora_refusals(kw, status):
    assert _lora(**kw) == status


def test_lora_plan_refusals():
    L = W.lib()
    assert L.w4a16_lora_plan(None, 4, 4, P, None) == W.ERR_NULL
    assert L.w4a16_lora_plan(P, 4, 4, None, None) == W.ERR_NULL
    assert L.w4a16_lora_plan(P, 4, 4, P + 8, None) == W.ERR_ALIGN
    assert L.w4a16_lora_plan(P, -1, 4, P, None) == W.ERR_SHAPE
    assert L.w4a16_lora_plan(P, 4, 1025, P, None) == W.ERR_SHAPE
    assert L.w4a16_lora_plan(None, 0, 4, None, None) == W.OK
    assert L.w4a16_lora_plan_bytes(4, 4, None) == W.ERR_NULL


def test_null_arguments():
    L = W.lib()
    assert L.w4a16_verify_drafts(None, None, 0, None) == W.ERR_NULL
    assert L.w4a16_lora(None, None, 0, None) == W.ERR_NULL
    for fn in (L.w4a16_pages_resize, L.w4a16_pages_fork, L.w4a16_kv_copy_pages, L.w4a16_kv_compact):
        assert fn(None, None) == W.ERR_NULL


def test_scratch_and_plan_sizes():
    # counters, then 16 bytes a chunk of 2048 and row, 24 a span of 1024 and sequence; those of a
    # row may start up to 7 logits before it
    assert scoring.verify_workspace_bytes(6, 2041, 2, 3, torch.bfloat16) == 65536 + 6 * 16 + 2 * 2 * 24
    assert scoring.verify_workspace_bytes(6, 2042, 2, 3, torch.bfloat16) == 65536 + 2 * 6 * 16 + 3 * 2 * 24
    assert scoring.verify_workspace_bytes(0, 2042, 2, 3, torch.float32) == 0
    # 4 bytes a tile, in whole 16, and 4 for each of its 16 or 64 rows
    assert adapters.plan_bytes(1, 4) == 16 + 64 and adapters.plan_bytes(0, 4) == 0
    assert adapters.plan_bytes(64, 32) == 4 * 36 + 4 * 16 * 36
    assert adapters.plan_bytes(640, 2) == 48 + 4 * 64 * 12
    # counters; for each of 16 rows the ranks (128 or 16 here) in two parts and a factor, and the sums of each split
    assert adapters.workspace_bytes(1, 128, 256, 4, 128) == 65536 + 16 * (128 + 1) * 4
    assert adapters.workspace_bytes(1, 20480, 256, 4, 8) > 65536 + 16 * (2 * 16 + 16 + 1) * 4
    # none where one kernel does both: 4 steps of k a wave, and up to 4096 columns each of 256 workgroups
    for rank, k in ((8, 8192), (16, 8192), (24, 4096), (32, 4096), (40, 2048), (64, 2048)):
        assert adapters.workspace_bytes(1, k, 256, 4, rank) == 0 != adapters.workspace_bytes(1, k + 8, 256, 4, rank)
    assert adapters.workspace_bytes(16, 512, 65536, 64, 16) == 0 != adapters.workspace_bytes(16, 512, 65544, 64, 16)
    assert adapters.workspace_bytes(257, 512, 256, 256, 16) != 0 == adapters.workspace_bytes(256, 512, 256, 256, 16)
    for bad in (dict(rank=7), dict(k=4), dict(tokens=-1), dict(adapters=0), dict(n=12)):
        with pytest.raises(W.W4A16Error):
            adapters.workspace_bytes(**{**dict(tokens=1, k=128, n=256, adapters=4, rank=8), **bad})


def test_cpu_tensors_are_refused():
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="same GPU"):
        adapters.lora_plan(z(3, **i32), 4)
    plan = adapters.LoraPlan(z(64, dtype=torch.uint8), 3, 4)
    with pytest.raises(ValueError, match="same GPU"):
        adapters.lora(z(3, 64).half(), z(4, 8, 64).half(), z(4, 32, 8).half(), plan)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        adapters.lora(z(3, 64), z(4, 8, 64), z(4, 32, 8), plan)
    with pytest.raises(ValueError, match="same GPU"):
        scoring.verify_drafts(z(2, 100), z(2, dtype=torch.int64), z(2, **i32), 2, z(2), z(1))
    with pytest.raises(ValueError, match="same GPU"):
        paging.cache_group([attn.kv_cache(2, 2, 64, 16, torch.float16, device="cpu")])
    with pytest.raises(ValueError, match="needs a cache"):
        paging.cache_group([])
    pool = paging.page_pool(4, 2, 3, 16, device="cpu")
    assert pool.refs.tolist() == [0] * 4 and pool.block_table.tolist() == [[-1] * 3] * 2
    for fn in (paging.pages_resize, paging.pages_fork):
        with pytest.raises(ValueError, match="same GPU"):
            fn(pool, z(1, **i32), z(1, **i32))


@pytest.mark.parametrize("name,count", [("table", 7 * 8 + 8), ("lens", 8), ("starts", 9), ("path", 8 * 4), ("counts", 8)])
@pytest.mark.parametrize("group", [1, 70])
def test_new_lengths_are_apart_from_what_is_read(name, count, group):
    # 8 sequences: arrays that end where the new lengths start, or start where those end, are apart
    at, size = 16 * P, dict(table=7 * 8 + 8, lens=8, starts=9, path=8 * 4, counts=8)
    call = lambda new: _compact([_cache()] * group, B=8, new=new,                                      # noqa: E731
                                **{n: at if n == name else 32 * P + i * P for i, n in enumerate(size)})
    for inside in (at, at + 4, at + 4 * (count - 1), at - 4 * 7):
        assert call(inside) == W.ERR_SHAPE and "new_lens" in W.last_error()
    if not HAS_GPU:
        assert call(at + 4 * count) == call(at - 4 * 8) == W.ERR_DEVICE


def test_arrays_of_no_entries_share_nothing():
    if not HAS_GPU:
        assert _compact(new=2 * P, path=2 * P, width=0) == _compact(new=2 * P, table=2 * P, entries=0) == W.ERR_DEVICE
