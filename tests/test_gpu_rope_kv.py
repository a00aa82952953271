"""GPU tests of rotary positions and the paged cache against the fp64 oracle.

Bounds: a 16-bit result is off by at most half a step, eps / 2 of its value (or
half the smallest subnormal), plus the fp32 arithmetic before it, at most 4
roundings of 2^-24 of the terms' magnitudes. A code is the nearest one to the
value in units of the scale, up to the fp32 error of that value: 8 roundings.
"""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as S
from weight_only_int4_unpack_amd import attn
from weight_only_int4_unpack_amd import w4a16 as W

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def say(*a):
    print(*a, flush=True)


def half_step16(y, dtype):
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2       # half a subnormal step
    return torch.finfo(dtype).eps / 2 * np.abs(y) + tiny


def f64(t):
    return t.detach().double().cpu().numpy()


def heads(shape, dtype, seed, pad=0):
    """Random heads; with `pad`, a view into wider rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, H, D = shape
    x = torch.randn((T, H + pad, D), generator=g, device="cuda").to(dtype)
    return x[:, pad // 2:pad // 2 + H] if pad else x


def table_of(positions, r, **kw):
    return attn.rope_table(positions, attn.rope_frequencies(r, 1e4, **kw))


def assert_rope(y, x, pos, table, inter, inverse=False):
    want = S.rope(f64(x), pos.cpu().numpy(), None, inter, inverse, table=f64(table))
    r = table.shape[1]
    x64 = f64(x)
    # |y| <= |x_a| + |x_b| <= the sum of the pair's magnitudes
    pair = np.abs(x64).copy()
    if inter:
        p = np.abs(x64[..., 0:r:2]) + np.abs(x64[..., 1:r:2])
        pair[..., 0:r:2] = pair[..., 1:r:2] = p
    else:
        p = np.abs(x64[..., :r // 2]) + np.abs(x64[..., r // 2:r])
        pair[..., :r // 2] = pair[..., r // 2:r] = p
    assert np.all(np.abs(f64(y) - want) <= half_step16(want, x.dtype) + 4 * U32 * pair * 2)
    assert torch.equal(y[..., r:], x[..., r:])


@pytest.mark.parametrize("positions,r,amp", [(1, 2, 1.0), (70001, 128, 1.0), (333, 80, 1.25), (17, 256, 1.0)])
def test_table(positions, r, amp):
    say("table", positions, r, amp)
    f = attn.rope_frequencies(r, 1e4)
    t = f64(attn.rope_table(positions, f, amp))
    a = np.arange(positions, dtype=np.float64)[:, None] * np.array(f)[None]
    want = amp * np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.all(np.abs(t - want) <= U32 * np.abs(want) + 1e-10)


ROPE = [  # tokens, heads, dim, rotated
    (1, 1, 8, 2), (1, 32, 128, 128), (5, 40, 128, 64), (7, 3, 80, 40), (3, 5, 80, 80), (9, 2, 96, 96),
    (2, 4, 256, 256), (2, 4, 256, 20), (33, 1, 64, 64), (4, 2, 72, 36), (257, 8, 128, 128), (3, 2, 40, 16),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,r", ROPE)
def test_rope(T, H, D, r, inter, dtype):
    say("rope", T, H, D, r, inter, dtype)
    x = heads((T, H, D), dtype, 1, pad=3)
    table = table_of(500, r)
    pos = torch.randint(0, 500, (T,), device="cuda")
    y = attn.rope(x, pos, table, interleaved=inter)
    assert_rope(y, x, pos, table, inter)
    back = attn.rope(x, pos, table, interleaved=inter, inverse=True)
    assert_rope(back, x, pos, table, inter, inverse=True)
    # in place, in a view of its own
    z = heads((T, H, D), dtype, 1, pad=3)
    assert attn.rope(z, pos, table, interleaved=inter, out=z) is z and torch.equal(z, y)


def test_rope_positions_outside_the_table_are_nan():
    x = heads((4, 2, 64), torch.bfloat16, 2)
    table = table_of(8, 32)
    pos = torch.tensor([-1, 7, 8, 2 ** 40], device="cuda")
    y = attn.rope(x, pos, table)
    assert torch.isnan(y[[0, 2, 3], :, :32]).all() and torch.equal(y[..., 32:], x[..., 32:])
    assert_rope(y[1:2], x[1:2], pos[1:2], table, False)


def test_rope_of_nothing():
    table = table_of(8, 32)
    for shape in [(0, 4, 64), (3, 0, 64)]:
        x = torch.empty(shape, dtype=torch.float16, device="cuda")
        assert attn.rope(x, torch.zeros(shape[0], dtype=torch.int64, device="cuda"), table).shape == shape


def slots_of(T, pages, page, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages * page, generator=g)[:T].cuda()


def dense(cache, slots):
    """Codes (and scales) of the given slots, fp64."""
    page = cache.k.shape[2]
    p, o = (slots // page).cpu(), (slots % page).cpu()
    out = []
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes = c.cpu().float().double()[p, :, o].numpy()
        out.append((codes, None if s is None else s.cpu().double()[p, :, o].numpy()))
    return out


def assert_written(x64, codes, scale, fmt, dtype, terms):
    """Codes [T, H, D] of values x64 computed in fp32 from `terms` magnitudes."""
    if fmt == "16":
        assert np.all(np.abs(codes - x64) <= half_step16(x64, dtype) + 8 * U32 * terms)
        return
    want = S.scale_of(x64, fmt)
    assert np.all(np.abs(scale - want) <= 8 * U32 * (want + terms.max(-1) / S.TOP[fmt]))
    unit = np.where(want > 0, want, 1.0)[..., None]
    y = x64 / unit
    slack = 8 * U32 * (np.abs(y) + terms / unit + S.TOP[fmt])
    step = np.maximum(S.half_step(np.abs(y) + slack, fmt), S.half_step(np.abs(codes), fmt))
    assert np.all(np.abs(codes - y) <= step + slack)


WRITE = [  # tokens, q heads, heads, dim, rotated, page
    (1, 4, 1, 64, 64, 16), (16, 40, 8, 128, 128, 64), (77, 8, 2, 80, 40, 32), (5, 4, 4, 256, 256, 128),
    (130, 7, 1, 96, 48, 16), (300, 32, 8, 128, 64, 64),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["16", "e4m3", "int8"])
@pytest.mark.parametrize("T,hq,hk,D,r,page", WRITE)
def test_kv_write(T, hq, hk, D, r, page, fmt, dtype):
    say("write", T, hq, hk, D, r, page, fmt, dtype)
    inter = (T + hq) % 2 == 0
    qkv = heads((T, hq + 2 * hk, D), dtype, 3)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pages = -(-T // page) + 2
    cache = attn.kv_cache(pages, hk, D, page, CODES.get(fmt, dtype))
    slots = slots_of(T, pages, page, 4)
    table = table_of(5000, r)
    pos = torch.randint(0, 5000, (T,), device="cuda")
    before = qkv.clone()
    qo = attn.kv_write(k, v, slots, cache, positions=pos, table=table, interleaved=inter, q=q)
    assert torch.equal(qkv, before)
    assert_rope(qo, q, pos, table, inter)
    k64 = S.rope(f64(k), pos.cpu().numpy(), None, inter, table=f64(table))
    v64 = f64(v)
    (kc, ks), (vc, vs) = dense(cache, slots)
    tk = np.abs(f64(k)).max(-1, keepdims=True) * np.ones_like(k64) * 2
    assert_written(k64, kc, ks, fmt, dtype, tk)
    assert_written(v64, vc, vs, fmt, dtype, np.abs(v64))
    # nothing else was written
    used = torch.zeros(pages * page, dtype=torch.bool)
    used[slots.cpu()] = True
    rest = (~used).nonzero().squeeze(1).cuda()
    for codes, scale in dense(cache, rest):
        assert not codes.any() and (scale is None or not scale.any())
    # read back: one rounding of code * scale
    rk, rv = attn.kv_read(cache, slots, dtype=dtype)
    for got, c, s in ((rk, kc, ks), (rv, vc, vs)):
        want = c if s is None else c * s[..., None]
        assert np.all(np.abs(f64(got) - want) <= half_step16(want, dtype) + U32 * np.abs(want))
    # without a rotation
    plain = attn.kv_cache(pages, hk, D, page, CODES.get(fmt, dtype))
    assert attn.kv_write(k, v, slots, plain) is None
    (kc, ks), _ = dense(plain, slots)
    assert_written(f64(k), kc, ks, fmt, dtype, np.abs(f64(k)))


@pytest.mark.parametrize("fmt", ["16", "e4m3", "int8"])
def test_slots_outside_the_cache(fmt):
    k, v = heads((5, 2, 64), torch.bfloat16, 5), heads((5, 2, 64), torch.bfloat16, 6)
    cache = attn.kv_cache(2, 2, 64, 16, CODES.get(fmt, torch.bfloat16))
    slots = torch.tensor([-1, 3, 32, -2 ** 60, 2 ** 60], device="cuda")
    attn.kv_write(k, v, slots, cache)
    inside = torch.arange(32, device="cuda")
    for codes, _ in dense(cache, inside):
        assert codes[3].any() and not np.delete(codes, 3, 0).any()
    rk, rv = attn.kv_read(cache, slots)
    assert rk[1].any() and not rk[[0, 2, 3, 4]].any() and not rv[[0, 2, 3, 4]].any()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_heads_of_zeros_tiny_and_non_finite(fmt):
    k = torch.zeros((6, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[1, 0, 5] = 2.0 ** -110                    # below the smallest head that is kept
    k[2, 0, 5] = 2.0 ** -90
    k[3, 0, 5] = float("inf")
    k[4, 0, 5] = float("nan")
    k[5, 0, :] = 3.0e38
    cache = attn.kv_cache(1, 1, 64, 16, CODES[fmt])
    slots = torch.arange(6, device="cuda")
    attn.kv_write(k, k, slots, cache)
    (codes, scale), _ = dense(cache, slots)
    assert not codes[:2].any() and not scale[:2].any()
    assert codes[2, 0, 5] == S.TOP[fmt] and scale[2, 0] > 0
    assert not codes[3:5].any() and np.isnan(scale[3:5]).all()
    assert (codes[5] == S.TOP[fmt]).all()
    rk, _ = attn.kv_read(cache, slots)
    assert torch.isnan(rk[3:5]).all() and not rk[:2].any()
    assert float(rk[5].float().min()) >= 2.97e38


def test_rounding_of_codes_is_to_nearest_even():
    # one head whose largest magnitude makes the scale 1: its values are the codes' grid
    for fmt in ("e4m3", "int8"):
        top = S.TOP[fmt]
        vals = [top, 2.5, 3.5, -2.5, 0.5, 1.5, 100.5, -top] if fmt == "int8" else \
            [top, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 432.0, -2.0 ** -11]
        want = [127, 2, 4, -2, 0, 2, 100, -127] if fmt == "int8" else \
            [448, 16, 20, -16, 0, 2.0 ** -8, 448, 0]
        k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
        k[0, 0, :8] = torch.tensor(vals, device="cuda")
        cache = attn.kv_cache(1, 1, 64, 16, CODES[fmt])
        attn.kv_write(k, k, torch.tensor([0], device="cuda"), cache)
        got = dense(cache, torch.tensor([0]))[0][0][0, 0, :8]
        assert got.tolist() == want, (fmt, got)


def test_every_code_reads_back():
    values = S.e4m3_values()
    for fmt in ("e4m3", "int8"):
        cache = attn.kv_cache(1, 1, 256, 16, CODES[fmt])
        cache.k.view(torch.uint8)[0, 0, 3] = torch.arange(256, dtype=torch.uint8, device="cuda")
        cache.k_scale.fill_(1.0)
        for dtype in (torch.float16, torch.bfloat16):
            rk, _ = attn.kv_read(cache, torch.tensor([3], device="cuda"), dtype=dtype)
            want = values if fmt == "e4m3" else np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)
            assert np.array_equal(f64(rk[0, 0]), want, equal_nan=True)


def test_refused_tensors():
    k = heads((4, 2, 64), torch.bfloat16, 7)
    cache = attn.kv_cache(2, 2, 64, 16)
    slots = torch.arange(4, device="cuda")
    for bad in (
        lambda: attn.kv_write(k, k[:3], slots, cache),
        lambda: attn.kv_write(k, k, slots.int(), cache),
        lambda: attn.kv_write(k, k, slots, cache._replace(k_scale=None)),
        lambda: attn.kv_write(k, k, slots, attn.kv_cache(2, 3, 64, 16)),
        lambda: attn.kv_write(k, k, slots, attn.kv_cache(2, 2, 64, 16, torch.float16)),
        lambda: attn.kv_write(k, k, slots, cache, q=k),
        lambda: attn.kv_write(k, k, slots, cache, positions=slots),
        lambda: attn.kv_write(k.transpose(1, 2), k, slots, cache),
        lambda: attn.kv_write(k.float(), k.float(), slots, cache),
        lambda: attn.kv_read(cache, slots.cpu()),
        lambda: attn.kv_read(cache, slots, dtype=torch.float32),
        lambda: attn.rope(k, slots, table_of(8, 64).half()),
        lambda: attn.rope(k, slots[:3], table_of(8, 64)),
        lambda: attn.rope(k[0], slots, table_of(8, 64)),
    ):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(W.W4A16Error) as e:     # rows 4 elements apart from 16-byte boundaries
        attn.rope(torch.zeros(4, 2, 68, dtype=torch.bfloat16, device="cuda")[..., 4:], slots, table_of(8, 64))
    assert e.value.status == W.ERR_ALIGN
    with pytest.raises(W.W4A16Error) as e:
        attn.rope(k, slots, table_of(8, 128))
    assert e.value.status == W.ERR_SHAPE


def test_offsets_past_4_gib():
    # 40000 pages x 8 heads x 64 tokens x 128 dims of bf16: 5.2 GB of keys
    cache = attn.KVCache(*[torch.empty((40000, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
                           for _ in range(2)])
    slots = torch.tensor([0, 39999 * 64 + 63, 38000 * 64 + 1], device="cuda")
    k, v = heads((3, 8, 128), torch.bfloat16, 8), heads((3, 8, 128), torch.bfloat16, 9)
    attn.kv_write(k, v, slots, cache)
    rk, rv = attn.kv_read(cache, slots)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    assert torch.equal(cache.k[39999, :, 63], k[1])
