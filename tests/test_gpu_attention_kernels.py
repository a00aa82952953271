"""GPU tests of every attention kernel (1 to 16, 17 to 32, 33 to 64 and more rows of a
key/value head, head dims of 64, 128, 256 and in between, each cache) with bounds in
which NaN fails: causal, trees, and trees with a sibling that holds infinities or NaN."""
import pytest
import torch

from attention_case import Strict
from test_gpu_tree_attention import ancestors, random_trees
from weight_only_int4_unpack_amd import attn

pytestmark = pytest.mark.gpu

FORMATS = [("16", torch.float16), ("16", torch.bfloat16), ("e4m3", torch.float16), ("e4m3", torch.bfloat16),
           ("int8", torch.float16), ("int8", torch.bfloat16)]
# new tokens of two sequences; with two query heads a key/value head twice as many rows
NEWS = [(1, 1), (4, 7), (10, 15), (16, 9), (20, 32), (25, 17), (40, 70)]


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [48, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("news", NEWS)
def test_causal_and_trees(news, dim, fmt, dtype):
    say("attention", news, dim, fmt, dtype)
    c = Strict([333, 130], list(news), 4, 2, dim, fmt, dtype, 32, seed=51)
    c.check(*c.run())
    trees = random_trees(news, 52)
    c.check(*c.run(mask=attn.tree_mask(trees)), rows=[ancestors(t) for t in trees])


@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_many_query_heads_of_a_key_head(fmt, dtype):
    # single tokens without masks, 17 to 32 rows
    for hq, dim in ((24, 128), (32, 64), (20, 80), (32, 256)):
        say("query heads", hq, dim, fmt, dtype)
        c = Strict([700, 33, 1, 250], [1, 1, 1, 1], hq, 1, dim, fmt, dtype, 64, seed=53)
        c.check(*c.run())


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("new", [4, 12, 24, 48])
def test_siblings_that_are_not_finite(new, dim, fmt, dtype, value):
    # drafted token 2 holds the value: seen by itself and what follows it, 3 and 5 (mod 6)
    say("not finite", new, dim, fmt, dtype, value)
    c = Strict([150, 61], [new, new], 4, 2, dim, fmt, dtype, 16, seed=54)
    parents = [-1, 0, 0, 2, 1, 3] + [j - 6 for j in range(6, new)]
    parents = parents[:new]
    rows = [ancestors(parents)] * 2
    hit = [i for i in range(new) if 2 in rows[0][i]]
    at = 150 - new + 2
    page, off = divmod(int(c.slots[0][at]), 16)
    for x, s in ((c.cache.k, c.cache.k_scale), (c.cache.v, c.cache.v_scale)):
        if s is None:
            x[page, :, off, 3] = value
        else:
            s[page, :, off] = value
            if fmt == "e4m3":
                x.view(torch.uint8)[page, :, off, 3] = 0x7F
    out, lse = c.run(mask=attn.tree_mask([parents] * 2))
    c.check(out, lse, rows=rows, which=[1])
    c.check(out, lse, rows=rows, which=[0], but=hit)
    assert hit and not bool(torch.isfinite(out[hit]).all(-1).any())


@pytest.mark.parametrize("news", [(1, 1), (10, 15), (20, 32), (40, 70)])
@pytest.mark.parametrize("fmt", ["16", "e4m3"])
def test_captured_with_eager_work_between(fmt, news):
    # every kernel in a graph on its first use in it, replayed as the cache changes
    say("captured", fmt, news)
    c = Strict([333, 130], list(news), 4, 2, 128, fmt, torch.bfloat16, 32, seed=55)
    k, v = (torch.randn((2, 2, 128), device="cuda").bfloat16() for _ in range(2))
    slots = torch.stack([c.slots[0][5], c.slots[1][-1]])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.kv_write(k, v, slots, c.cache)
        out, lse = c.run()
    for seed in range(3):
        for x in (k, v):
            x.copy_(torch.randn((2, 2, 128), device="cuda"))
        graph.replay()
        want = c.run()                          # eager, on the same stream
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        c.check(out, lse)
