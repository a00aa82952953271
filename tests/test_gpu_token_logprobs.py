"""GPU tests of token log probabilities against the fp64 oracle.

Bound: a sum of n positive fp32 terms of relative error e each is off by at most
(n + e) roundings; a thread adds up to V / 256 + 32 terms in turn and the joins
add 16 more, and a term e^d carries |d| + 2 roundings, of which e^d |d| <= 1
counts against the largest term. So ln(sum) is off by at most
(V / 256 + 64) 2^-24 =: s, a log probability by that and 2 roundings of its own
size and the maximum's, and the entropy by 4 s (1 + the entropy).
"""
import numpy as np
import pytest
import torch

from oracle import serve_oracle as S
from weight_only_int4_unpack_amd import scoring
from weight_only_int4_unpack_amd import w4a16 as W

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def say(*a):
    print(*a, flush=True)


def check(x, ids, k):
    """`x` on the GPU, finite maximum and no NaN in each row."""
    T, V = x.shape
    lp, H, top, at = scoring.token_logprobs(x, ids, k)
    assert lp.shape == H.shape == (T,) and top.shape == at.shape == (T, k)
    x64 = x.detach().double().cpu().numpy()
    wlp, wH, wtop, wat = S.token_logprobs(x64, ids.cpu().numpy(), k)
    assert np.array_equal(at.cpu().numpy(), wat)
    s = (V / 256 + 64) * U32

    def near(a, b, extra):
        a, b = a.double().cpu().numpy(), np.asarray(b)
        fine = np.isfinite(b)
        assert np.array_equal(np.isfinite(a), fine) and np.array_equal(a[~fine], b[~fine])
        assert np.all(np.abs(a[fine] - b[fine]) <= (s + 4 * U32 * np.abs(b) + extra)[fine])

    near(lp, wlp, np.zeros(T))
    near(top, wtop, np.zeros((T, k)))
    near(H, wH, 4 * s * (1 + wH))
    return lp, H, top, at


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,k", [
    (1, 1, 1), (1, 2, 0), (3, 63, 5), (2, 257, 32), (1, 8191, 20), (5, 8192, 20), (2, 8193, 33),
    (4, 32000, 5), (1, 100003, 64), (7, 50257, 20), (300, 1000, 3), (1, 600001, 20),
])
def test_sizes(T, V, k, dtype):
    say("score", T, V, k, dtype)
    g = torch.Generator(device="cuda").manual_seed(T * V + k)
    x = (torch.randn((T, V), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    a = check(x, ids, k)
    b = scoring.token_logprobs(x, ids, k)        # the same again, bit for bit
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("order", ["ascending", "descending", "equal", "two", "steps"])
def test_orders_that_fill_the_list(order, dtype):
    # ascending logits pass every earlier bound; equal ones are all ties
    V = 40000
    n = torch.arange(V, device="cuda")
    x = {"ascending": n / 1000.0, "descending": -n / 1000.0, "equal": n * 0.0,
         "two": (n % 2) * 1.0, "steps": (n // 5000) * 1.0}[order]
    x = x.to(dtype).repeat(3, 1).contiguous()
    for k in (1, 20, 64):
        say("order", order, dtype, k)
        check(x, torch.tensor([0, 17, V - 1], device="cuda"), k)


def test_rows_apart_and_unaligned():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((6, 20011), generator=g, device="cuda").to(torch.bfloat16)
    for lo, hi in [(0, 20011), (1, 20011), (3, 8195), (5, 16390), (7, 8), (9, 9010)]:
        say("columns", lo, hi)
        x = wide[::2, lo:hi]
        check(x, torch.zeros(3, dtype=torch.int64, device="cuda"), min(4, hi - lo))


def test_masked_vocabulary():
    # fewer allowed tokens than alternatives: -inf ones follow by lowest index
    x = torch.full((3, 30000), -float("inf"), device="cuda")
    x[0, [7, 29999, 8]] = torch.tensor([1.0, 2.0, 2.0], device="cuda")
    x[1, 12345] = -4.0
    x[2, :] = 0.25
    x[2, 100:] = -float("inf")
    lp, H, top, at = check(x, torch.tensor([7, 0, 99], device="cuda"), 6)
    assert at[0].tolist() == [8, 29999, 7, 0, 1, 2] and at[1].tolist()[:3] == [12345, 0, 1]
    assert float(lp[1]) == -float("inf") and float(H[1]) == 0.0


def test_rows_without_a_softmax():
    V = 20000
    x = torch.randn((5, V), device="cuda")
    x[0, 9000] = float("nan")
    x[1, 3] = float("inf")
    x[2, :] = -float("inf")
    x[3, :] = float("nan")
    lp, H, top, at = scoring.token_logprobs(x, torch.zeros(5, dtype=torch.int64, device="cuda"), 8)
    assert torch.isnan(lp[:4]).all() and torch.isnan(H[:4]).all() and torch.isnan(top[:4]).all()
    assert torch.isfinite(lp[4]) and torch.isfinite(H[4]) and torch.isfinite(top[4]).all()
    at = at.cpu().numpy()
    assert ((at >= 0) & (at < V)).all() and all(len(set(r)) == 8 for r in at)
    assert at[1][0] == 3 and 9000 not in at[0] and at[2].tolist() == list(range(8))


def test_ids_outside_the_vocabulary():
    x = torch.randn((4, 500), device="cuda").half()
    ids = torch.tensor([-1, 0, 500, 2 ** 40], device="cuda")
    lp, H, _, _ = scoring.token_logprobs(x, ids)
    assert torch.isnan(lp[[0, 2, 3]]).all() and torch.isfinite(lp[1]) and torch.isfinite(H).all()


def test_large_values_and_signed_zeros():
    x = torch.zeros((2, 9000), device="cuda")
    x[0, 5:] = -0.0                                  # +0 and -0 are one value: lowest index first
    x[1] = 60000.0
    x[1, 7] = 60004.0
    check(x, torch.tensor([8999, 7], device="cuda"), 8)
    assert scoring.token_logprobs(x, torch.tensor([0, 0], device="cuda"), 8)[3][0].tolist() == list(range(8))


def test_nothing_and_refusals():
    empty = scoring.token_logprobs(torch.empty((0, 50), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0, 3), (0, 3)]
    x = torch.zeros((2, 50), device="cuda")
    ids = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (lambda: scoring.token_logprobs(x.double(), ids), lambda: scoring.token_logprobs(x, ids.int()),
                lambda: scoring.token_logprobs(x, ids[:1]), lambda: scoring.token_logprobs(x.t(), ids),
                lambda: scoring.token_logprobs(x[0], ids)):
        with pytest.raises(ValueError):
            bad()
    for k in (-1, 51, 65):
        with pytest.raises(W.W4A16Error):
            scoring.token_logprobs(x, ids, k)


def test_captured_and_on_another_stream():
    x = torch.randn((5, 70000), device="cuda").bfloat16()
    ids = torch.randint(0, 70000, (5,), device="cuda")
    want = scoring.token_logprobs(x, ids, 10)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        got = scoring.token_logprobs(x, ids, 10)
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = scoring.token_logprobs(x, ids, 10)
    for seed in range(3):
        x.copy_(torch.randn((5, 70000), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = scoring.token_logprobs(x, ids, 10)
        assert all(torch.equal(a, b) for a, b in zip(held, want))
