"""GPU tests of attention over the paged cache against the fp64 oracle.

Bounds, for out = sum p v / sum p with mean magnitude A = sum p |v| / sum p:
  * a weight is rounded to 16 bits: at most half a step, eps / 2 relative
    (bf16 in front of 8-bit codes), so eps_p / 2 of A;
  * a score is a sum of D products in fp32 and two multiplications: off by at
    most (D + 4) 2^-24 of B = max |scale| sum |q k|, and e^s by that relative
    (and 2^-22 (|s| + 4) of exp2 and its argument, |s| <= B); in numerator and
    denominator, so twice;
  * N additions in fp32: N 2^-24 of A, numerator and denominator, so twice;
  * the result is rounded: eps / 2 of it. fp16 weights have a floor of 2^-31 of
    the largest weight each: N 2^-30 of the largest |v|.
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


class Case:
    """Random sequences in a paged cache, and dense fp64 copies of them."""

    def __init__(self, lens, news, hq, hk, D, fmt="16", dtype=torch.bfloat16, page=64, seed=0, sharp=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.news, self.fmt, self.dtype, self.page = lens, news, fmt, dtype, page
        self.hq, self.hk, self.D = hq, hk, D
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").int().cpu()
        width = max(need + [1])
        table = torch.full((len(lens), width), -7, dtype=torch.int32)     # past the end: no page
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table.cuda()
        self.cache = attn.kv_cache(pages, hk, D, page, CODES.get(fmt, dtype))
        # stale slots hold what must not be met: NaN
        if fmt == "16":
            self.cache.k.fill_(float("nan"))
            self.cache.v.fill_(float("nan"))
        else:
            self.cache.k.view(torch.uint8).fill_(0x7F)
            self.cache.v.view(torch.uint8).fill_(0x7F)
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("nan"))
        self.slots = [torch.tensor([int(table[b, t // page]) * page + t % page for t in range(n)],
                                   dtype=torch.int64, device="cuda") for b, n in enumerate(lens)]
        k = torch.randn((sum(lens), hk, D), generator=g, device="cuda").to(dtype)
        v = torch.randn((sum(lens), hk, D), generator=g, device="cuda").to(dtype)
        slots = torch.cat(self.slots) if lens else torch.empty(0, dtype=torch.int64, device="cuda")
        attn.kv_write(k, v, slots, self.cache)
        self.q = (torch.randn((sum(news), hq, D), generator=g, device="cuda") * sharp).to(dtype)
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.starts = torch.from_numpy(starts).cuda()
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5

    def dense(self, b):
        """fp64 keys and values of sequence b as the cache holds them."""
        out = []
        s = self.slots[b].cpu()
        for c, sc in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            x = c.cpu().float().double()[s // self.page, :, s % self.page].numpy()
            if sc is not None:
                x = x * sc.cpu().double()[s // self.page, :, s % self.page].numpy()[..., None]
            out.append(x)
        return out

    def run(self, mask=None, **kw):
        return attn.tree_attention(self.q, self.cache, self.table, self.kv_lens, self.starts,
                                   max(self.news + [1]), mask=mask, **{"scale": self.scale, **kw})

    def check(self, out, lse, parents=None, rows=None, which=None):
        eps16 = torch.finfo(self.dtype).eps / 2
        epsp = eps16 if self.fmt == "16" else 2.0 ** -8
        at = 0
        for b, (length, n) in enumerate(zip(self.lens, self.news)):
            if n == 0 or (which is not None and b not in which):
                at += n
                continue
            see = S.tree_visible(length, n, None if rows is None else rows[b])
            q = self.q[at:at + n].double().cpu().numpy()
            k, v = self.dense(b)
            want, wlse, A, B = S.attention(q, k, v, see, self.scale)
            got = out[at:at + n].double().cpu().numpy()
            glse = lse[at:at + n].double().cpu().numpy()
            N = length + 64
            score = (self.D + 4) * U32 * B + 2.0 ** -22 * (B + 4)
            big = max([np.abs(v).max()] if v.size else [0.0])
            tol = (epsp + 2 * score[..., None] + 2 * N * U32) * A + eps16 * np.abs(want) + \
                N * 2.0 ** -30 * big + torch.finfo(self.dtype).tiny
            bad = np.abs(got - want) > tol
            assert not bad.any(), (b, int(bad.sum()), float((np.abs(got - want) / tol).max()))
            assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
            fine = np.isfinite(wlse)
            ltol = score + N * U32 + 4 * U32 * np.abs(np.where(fine, wlse, 0))
            assert np.all(np.abs(glse[fine] - wlse[fine]) <= ltol[fine])
            at += n


def ancestors(parents):
    rows = []
    for j, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else frozenset()) | {j})
    return rows


def random_trees(news, seed):
    rng = np.random.default_rng(seed)
    return [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for n in news]


SHAPES = [  # lens, news, q heads, heads, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([300], [1], 8, 2, 128, 64),
    ([31, 32, 33, 127, 128, 129, 0, 1], [1, 1, 1, 1, 1, 1, 0, 1], 4, 1, 128, 16),
    ([700, 5, 260], [3, 5, 1], 10, 2, 80, 32),
    ([513, 90], [17, 17], 8, 8, 96, 64),
    ([1029, 64], [30, 1], 14, 2, 64, 128),
    ([400, 33], [2, 9], 4, 2, 256, 64),
    ([200], [70], 5, 1, 128, 64),
    ([150, 80], [150, 80], 2, 1, 128, 32),
    ([77], [20], 3, 1, 16, 16),
    ([90], [4], 6, 2, 144, 16),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["16", "e4m3", "int8"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_causal_and_trees(shape, fmt, dtype):
    lens, news, hq, hk, D, page = SHAPES[shape]
    say("attention", SHAPES[shape], fmt, dtype)
    c = Case(lens, news, hq, hk, D, fmt, dtype, page, seed=shape)
    out, lse = c.run()
    c.check(out, lse)
    trees = random_trees(news, shape)
    out, lse = c.run(mask=attn.tree_mask(trees))
    c.check(out, lse, rows=[ancestors(t) for t in trees])


@pytest.mark.parametrize("dim", [8, 24, 72, 120, 40])
def test_odd_head_dims(dim):
    say("dim", dim)
    c = Case([100, 45], [3, 20], 4, 2, dim, "16", torch.float16, 16, seed=dim)
    c.check(*c.run())


def test_long_contexts_are_split():
    # one long sequence among short ones; more splits than lanes
    c = Case([9000, 3, 40], [2, 1, 1], 4, 1, 64, "int8", torch.bfloat16, 16, seed=5, sharp=4.0)
    c.check(*c.run())
    again = c.run()
    assert all(torch.equal(a, b) for a, b in zip(again, c.run()))   # bit for bit


def test_more_sequences_than_lanes():
    lens = [(37 * b) % 200 for b in range(150)]
    news = [min(n, 1 + b % 3) for b, n in enumerate(lens)]
    c = Case(lens, news, 4, 2, 64, "e4m3", torch.bfloat16, 16, seed=6)
    c.check(*c.run())


def test_rows_that_see_nothing():
    # a mask of zeros, and no cached tokens before the new ones
    c = Case([5, 70], [5, 3], 4, 2, 64, "16", torch.bfloat16, 16, seed=7)
    mask = torch.zeros((8, 1), dtype=torch.int64, device="cuda")
    mask[2, 0] = 0b11000
    out, lse = c.run(mask=mask)
    rows = [[set(), set(), {3, 4}, set(), set()], [set()] * 3]
    c.check(out, lse, rows=rows)
    assert not out[[0, 1, 3, 4]].any() and torch.isneginf(lse[[0, 1, 3, 4]]).all()
    # sequences of no cached tokens, fewer cached than new ones, and a negative length
    c.kv_lens.copy_(torch.tensor([0, -5], dtype=torch.int32))
    out, lse = c.run()
    assert not out.any() and torch.isneginf(lse).all()
    c.kv_lens.copy_(torch.tensor([2, 70], dtype=torch.int32))
    out, lse = c.run()                       # new token i is cached token i - 3
    assert not out[:3].any() and torch.isneginf(lse[:3]).all() and torch.isfinite(lse[3:]).all()


def test_infinities_and_nan_in_masked_places():
    # drafted siblings: a non-finite value in one must not reach the others
    for value in (float("inf"), float("nan"), -float("inf")):
        for fmt, dtype in (("16", torch.bfloat16), ("16", torch.float16), ("int8", torch.bfloat16),
                           ("e4m3", torch.float16)):
            say("non-finite", value, fmt, dtype)
            c = Case([90, 40], [6, 6], 4, 2, 64, fmt, dtype, 16, seed=8)
            trees = [[-1, 0, 0, 1, 1, 2]] * 2
            rows = [ancestors(t) for t in trees]
            mask = attn.tree_mask(trees)
            want, wlse = c.run(mask=mask)
            slot = int(c.slots[0][90 - 6 + 2])       # node 2: seen by itself and node 5
            page, off = slot // 16, slot % 16
            for x, s in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)):
                if fmt == "16":
                    x[page, :, off, 3] = value
                else:
                    s[page, :, off] = value
                    if fmt == "e4m3":
                        x.view(torch.uint8)[page, :, off, 3] = 0x7F
            out, lse = c.run(mask=mask)
            others = [0, 1, 3, 4] + list(range(6, 12))
            assert torch.isfinite(out[others]).all()
            eps = torch.finfo(dtype).eps          # another order of products: a step at most
            assert torch.allclose(out[others].float(), want[others].float(), rtol=2 * eps, atol=2 * eps)
            assert torch.equal(lse[others], wlse[others])
            assert not torch.isfinite(out[[2, 5]]).all()
            c.check(want, wlse, rows=rows)


def test_masks_past_64_tokens_and_extra_words():
    news = [70, 130]
    trees = random_trees(news, 3)
    c = Case([200, 131], news, 2, 1, 64, "16", torch.float16, 32, seed=9)
    mask = attn.tree_mask(trees)
    assert mask.shape[1] == 3
    out, lse = c.run(mask=mask)
    c.check(out, lse, rows=[ancestors(t) for t in trees])
    wide = torch.cat([mask, torch.full((200, 2), -1, dtype=torch.int64, device="cuda")], 1)
    again = c.run(mask=wide)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_pages_and_lengths_outside():
    c = Case([100, 100], [1, 1], 4, 2, 64, "16", torch.bfloat16, 16, seed=10)
    good, _ = c.run()
    table = c.table.clone()
    table[0, 2] = -1                            # tokens 32..47 of sequence 0 lie nowhere
    table[0, 4] = 1 << 30
    bad = c.table.clone()
    c.table = table
    out, lse = c.run()
    keep = [t for t in range(100) if t // 16 not in (2, 4)]
    k, v = c.dense(0)
    want, wlse, _, _ = S.attention(c.q[:1].double().cpu().numpy(), k[keep], v[keep],
                                   np.ones((1, len(keep)), bool), c.scale)
    assert np.allclose(out[:1].double().cpu().numpy(), want, rtol=2 ** -7, atol=2 ** -7)
    assert np.allclose(lse[:1].double().cpu().numpy(), wlse, atol=1e-4)
    assert torch.equal(out[1], good[1])
    # a length past the table counts what the table holds
    c.table = bad
    c.kv_lens.copy_(torch.tensor([1 << 30, 100], dtype=torch.int32))
    out, _ = c.run()
    assert torch.equal(out[1], good[1])
    # rows past max_q are not computed; starts outside are cut
    c.starts.copy_(torch.tensor([0, 1, 1 << 30], dtype=torch.int32))
    out, _ = c.run()
    assert torch.equal(out[1], good[1])


def test_an_empty_cache():
    cache = attn.kv_cache(0, 2, 64, 16)
    q = torch.randn((3, 4, 64), device="cuda").bfloat16()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = attn.tree_attention(q, cache, torch.zeros((1, 4), dtype=torch.int32, device="cuda"), ints(50),
                                   ints(0, 3), 3)
    assert not out.any() and torch.isneginf(lse).all()


def test_views_scales_and_streams():
    c = Case([300, 77], [2, 5], 8, 2, 128, "e4m3", torch.bfloat16, 64, seed=11)
    out, lse = c.run()
    wide = torch.randn((7, 12, 128), device="cuda").bfloat16()
    wide[:, 2:10] = c.q
    c.q = wide[:, 2:10]
    again = c.run(out=torch.empty_like(out), lse=torch.empty_like(lse))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    c.table = torch.cat([c.table, c.table], 1)[:, :c.table.shape[1]]          # rows apart
    assert torch.equal(c.run()[0], out)
    for scale in (-0.3, 0.0, 1e-3, 3.0):
        say("scale", scale)
        c.scale = scale
        c.check(*c.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], c.run()[0])


@pytest.mark.parametrize("fmt", ["16", "e4m3"])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_a_scale_of_zero_and_negative_ones(new, fmt):
    for scale in (0.0, -0.0, -0.4):
        say("scale", scale, new, fmt)
        c = Case([70, 41], [new, new], 8, 2, 64, fmt, torch.bfloat16, 16, seed=21)
        c.scale = scale
        c.check(*c.run())
        if new > 1:
            trees = random_trees([new, new], 4)
            c.check(*c.run(mask=attn.tree_mask(trees)), rows=[ancestors(t) for t in trees])


def test_captured_launch_follows_the_lengths():
    c = Case([900, 333], [3, 3], 8, 2, 64, "int8", torch.float16, 16, seed=12)
    mask = attn.tree_mask([[-1, 0, 0]] * 2)
    c.run(mask=mask)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run(mask=mask)
    for lens in ([900, 333], [3, 200], [500, 3], [900, 333]):
        say("replay", lens)
        c.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = c.run(mask=mask)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_offsets_past_4_gib():
    # pages at the end of a cache of 5.2 GB of keys
    cache = attn.KVCache(*[torch.zeros((40000, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
                           for _ in range(2)])
    k, v = (torch.randn((100, 8, 128), device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[39999, 39000]], dtype=torch.int32, device="cuda")
    t = torch.arange(100, device="cuda")
    attn.kv_write(k, v, table[0].long()[t // 64] * 64 + t % 64, cache)
    q = torch.randn((1, 32, 128), device="cuda").bfloat16()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, _ = attn.tree_attention(q, cache, table, ints(100), ints(0, 1), 1)
    want, _, A, _ = S.attention(q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                np.ones((1, 100), bool), 128 ** -0.5)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2 ** -7 * (A + np.abs(want)))


def test_refused_tensors():
    c = Case([50], [2], 4, 2, 64, "16", torch.bfloat16, 16, seed=13)
    args = dict(q=c.q, cache=c.cache, block_table=c.table, kv_lens=c.kv_lens, q_starts=c.starts, max_q=2)
    for kw in (dict(q=c.q.half()), dict(q=c.q[:, :3]), dict(block_table=c.table.long()), dict(kv_lens=c.kv_lens.long()),
               dict(q_starts=c.starts[:1]), dict(mask=torch.zeros((2, 1), dtype=torch.int32, device="cuda")),
               dict(mask=torch.zeros((3, 1), dtype=torch.int64, device="cuda")), dict(out=c.q.float()),
               dict(kv_lens=c.kv_lens.cpu()), dict(cache=attn.kv_cache(2, 2, 128, 16, torch.bfloat16))):
        with pytest.raises(ValueError):
            attn.tree_attention(**{**args, **kw})
    with pytest.raises(W.W4A16Error) as e:
        attn.tree_attention(**args, scale=float("nan"))
    assert e.value.status == W.ERR_VALUE
