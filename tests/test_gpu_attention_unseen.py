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
