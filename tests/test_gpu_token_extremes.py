"""GPU tests of token scores at the ends of the types: tokens masked by the lowest
finite value, rows of nothing else, and logits near the largest. Bounds as in
``test_gpu_token_logprobs``; a difference of two logits that fp32 cannot hold is
-infinity."""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as S
from test_gpu_token_logprobs import DTYPES, U32
from weight_only_int4_unpack_amd import scoring

pytestmark = pytest.mark.gpu


def check(x, ids, k):
    lp, H, top, at = scoring.token_logprobs(x, ids, k)
    with np.errstate(over="ignore"):
        wlp, wH, wtop, wat = S.token_logprobs(x.double().cpu().numpy(), ids.cpu().numpy(), k)
        s = (x.shape[1] / 256 + 64) * U32
        assert np.array_equal(at.cpu().numpy(), wat)
        for got, want, extra in ((lp, wlp, 0.0), (top, wtop, 0.0), (H, wH, 4 * s * (1 + wH))):
            got = got.double().cpu().numpy()
            held = want.astype(np.float32).astype(np.float64)       # -inf past fp32's range
            fine = np.isfinite(held)
            assert np.array_equal(got[~fine], held[~fine])
            assert np.all(np.abs(got - want)[fine] <= np.broadcast_to(s + 4 * U32 * np.abs(want) + extra, want.shape)[fine])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [9, 8191, 32000, 100003])
def test_tokens_masked_by_the_lowest_value(V, dtype):
    print("masked", V, dtype, flush=True)
    low = torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn((6, V), generator=g, device="cuda") * 3).to(dtype)
    x[0, 1:] = low                                # one token allowed
    x[1, ::2] = low
    x[2, V // 2:] = low                           # whole parts
    x[3, :] = low                                 # none: all alike
    x[4, :] = low
    x[4, V - 1] = low / 2                         # one far above the rest, and far below 0
    x[5, 0] = low
    ids = torch.tensor([V - 1, 0, V - 1, 3, V - 1, 0], device="cuda")
    for k in (0, 5, 9):
        check(x, ids, k)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logits_near_the_largest(dtype):
    big = torch.finfo(dtype).max
    x = torch.zeros((5, 20000), device="cuda", dtype=dtype)
    x[0, 7] = big
    x[1, :] = big
    x[2, [3, 19999]] = big
    x[3, :] = -big
    x[3, 5] = big                                 # differences past fp32's range
    x[4, :] = big
    x[4, 100:] = -big
    check(x, torch.tensor([7, 19, 3, 5, 0], device="cuda"), 8)
    check(x, torch.tensor([0, 0, 0, 6, 19999], device="cuda"), 64)
