"""GPU tests: large values in tokens that a row does not see, or gives no weight,
leave the row what it is."""
import pytest
import torch

from attention_case import Strict
from test_gpu_tree_attention import ancestors
from weight_only_int4_unpack_amd import attn

pytestmark = pytest.mark.gpu

NEWS = [4, 10, 20, 40]          # 8, 20, 40 and 80 rows: each kernel


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", NEWS)
def test_a_nan_scale_beside_a_larger_finite_one(new, dim):
    # Each drafted token sees the cached ones and itself. One lane holds tokens
    # 868..871: 870's scale is NaN, 871's V 2^20 times as large as all before it. So
    # many sequences that a wave meets other tokens first.
    say("NaN beside", new, dim)
    n = 64
    c = Strict([872] * n, [new] * n, 4, 2, dim, "e4m3", torch.bfloat16, 16, seed=31)
    mask = attn.tree_mask([[-1] * new] * n)
    for b in range(n):
        c.multiply_v(b, 871, 2.0 ** 20)
    want, wlse = c.run(mask=mask)
    for b in range(n):
        c.values(b, 870)[1].fill_(float("nan"))
    out, lse = c.run(mask=mask)
    each = torch.arange(n * new, device="cuda") % new
    assert torch.isnan(out[each == new - 2]).all()
    keep = each != new - 2
    assert bool(torch.isfinite(out[keep]).all())
    # the same weights against another power of two: at most a step of the output
    assert torch.allclose(out[keep].float(), want[keep].float(), rtol=2 ** -7, atol=2 ** -7)
    assert torch.equal(lse[keep], wlse[keep])


@pytest.mark.parametrize("value", [1e6, 1e10, 1e30])
@pytest.mark.parametrize("fmt,dim", [("e4m3", 64), ("e4m3", 128), ("e4m3", 256), ("int8", 128), ("16", 128)])
@pytest.mark.parametrize("new", NEWS)
def test_large_finite_siblings(new, fmt, dim, value):
    # a garbage draft: seen by itself alone, in the tile of all the others
    say("large sibling", new, fmt, dim, value)
    c = Strict([90, 300], [new, new], 4, 2, dim, fmt, torch.bfloat16, 16, seed=32)
    trees = [[-1, 0, 0] + [1] * (new - 3)] * 2
    for b, length in enumerate(c.lens):
        x = torch.full((1, 2, dim), value, dtype=torch.bfloat16, device="cuda")
        k = torch.randn((1, 2, dim), device="cuda").bfloat16()
        attn.kv_write(k, x, c.slots[b][length - new + 2:length - new + 3], c.cache)
    rows = [ancestors(t) for t in trees]
    c.check(*c.run(mask=attn.tree_mask(trees)), rows=rows)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("new,value", [(1, 1e10), (1, 1e20), (10, 1e10), (20, 1e10), (40, 1e10)])
@pytest.mark.parametrize("at", [0, 40, 250])
def test_large_values_without_weight(at, new, value, fmt):
    # a token that rows see and whose score lies far below the others': e^-60 times 1e10
    # (1e20) is small beside their values of about 1
    say("no weight", at, new, value, fmt)
    c = Strict([300], [new], 2, 2, 128, fmt, torch.bfloat16, 16, seed=33)
    c.q[:] = c.q[:1]                                    # one query for all rows of a head
    k = -2.0 * c.q[:1] * 2.0 ** torch.round(torch.log2(30.0 / (c.scale * (c.q[:1].float() ** 2).sum(-1, keepdim=True))))
    x = torch.full((1, 2, 128), value, dtype=torch.bfloat16, device="cuda")
    attn.kv_write(k.bfloat16(), x, c.slots[0][at:at + 1], c.cache)
    c.check(*c.run())
