"""GPU tests of low-rank adapters beside a shared product, against the fp64 oracle.

Tolerance of one output y = base + s sum_r v_r b_r, v_r = sum_k x_k a_k, by element:
the products of v are exact in fp32 or rounded by 2^-24, and of K sums each rounds by at
most 2^-24 of the sum of magnitudes: K 2^-23 sum |x a| covers both; v in two 16-bit
parts is off by 2^-18 (bf16: 9 and 9 bits, rounding each by half a step) or 2^-22 (fp16;
below 2^-39 of a row's largest v nothing is held, 2^-38 max|v| |b| covers it); the sum over
2 R products by 2 R 2^-23; the last addition by 2^-23 of both sides; the result by half a
step of its type, eps / 2, and below the smallest normal number by half of the smallest
subnormal one."""
import math

import numpy as np
import pytest
import torch

from oracle import batch_oracle as O
from weight_only_int4_unpack_amd import adapters

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(seed, T, K, N, R, rank, dtype="bf16", index=None, ranks=None, scales=True, base=True, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)                                   # noqa: E731
    dt = DT[dtype]
    n = np.random.default_rng(seed)
    return dict(x=rand(T, K).to(dt), a=(rand(R, rank, K) * gain / math.sqrt(K)).to(dt),
                b=(rand(R, N, rank) / gain / math.sqrt(rank)).to(dt), base=rand(T, N).to(dt) if base else None,
                index=n.integers(-1, R, T).tolist() if index is None else index, ranks=ranks,
                scales=(torch.rand((R,), generator=g) + 0.5) * torch.tensor([1.0, -1.0])[torch.arange(R) % 2] if scales else None)


def run(c, plan=None, **kw):
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    plan = plan or adapters.lora_plan(ints(c["index"]), c["a"].shape[0])
    a = dict(base=dev["base"], scales=dev["scales"], ranks=None if c["ranks"] is None else ints(c["ranks"]))
    a.update(kw)
    return adapters.lora(dev["x"], dev["a"], dev["b"], plan, **a)


def f64(t):
    return None if t is None else t.double().numpy()


def check(got, c, rows=None):
    y, vb, deep = O.lora(f64(c["x"]), f64(c["a"]), f64(c["b"]), c["index"], f64(c["base"]), f64(c["scales"]), c["ranks"])
    dt, K, rank = c["x"].dtype, c["x"].shape[1], c["a"].shape[1]
    info = torch.finfo(dt)
    split = 2.0 ** -18 if dt == torch.bfloat16 else 2.0 ** -22
    # a row's largest |v| against |b|, for fp16's smallest parts
    small = 0.0 if dt == torch.bfloat16 else 2.0 ** -38 * vb.max(-1, keepdims=True) * rank
    base = 0.0 if c["base"] is None else np.abs(f64(c["base"]))
    tol = (deep * K * 2.0 ** -23 + vb * (split + 2 * rank * 2.0 ** -23) + small + (base + vb) * 2.0 ** -23)
    tol = tol + info.eps / 2 * (np.abs(y) + tol) + info.smallest_normal * info.eps / 2
    off = np.abs(got.double().cpu().numpy() - y)
    rows = slice(None) if rows is None else rows
    bad = off[rows] > tol[rows]
    assert not bad.any(), (int(bad.sum()), float((off[rows] / tol[rows]).max()))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("T,K,N,R", [(1, 8, 8, 1), (3, 136, 72, 2), (17, 1000, 264, 3), (64, 2112, 1032, 5),
                                     (200, 520, 336, 2), (300, 4096, 128, 3)])
def test_against_the_oracle(T, K, N, R, rank, dtype):
    c = make(T + rank, T, K, N, R, rank, dtype)
    check(run(c), c)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("T,K,N,R,rank", [(1, 8192, 136, 2, 8), (1, 8200, 136, 2, 8), (40, 8192, 1032, 4, 16),
                                          (40, 8200, 1032, 4, 16), (5, 4096, 520, 1, 32), (5, 4104, 520, 1, 32),
                                          (3, 2048, 4104, 2, 64), (3, 2056, 4104, 2, 64), (100, 264, 8200, 30, 16),
                                          (200, 264, 12320, 64, 16), (200, 264, 12296, 64, 16), (200, 264, 12320, 64, 32),
                                          (200, 264, 8192, 64, 64), (300, 72, 264, 255, 24), (255, 72, 264, 255, 24),
                                          (9, 40000, 72, 9, 48)])
def test_one_kernel_or_two(T, K, N, R, rank, dtype):
    # around the sizes from which on the two products are launched apart
    c = make(K, T, K, N, R, rank, dtype)
    got = run(c)
    check(got, c)
    base = c["base"].cuda()
    assert torch.equal(run(c, base=base, out=base), got) and torch.equal(base, got)


@pytest.mark.parametrize("rank", [8, 32, 64, 128])
@pytest.mark.parametrize("T,R,N", [(64, 64, 8200), (64, 64, 16392), (64, 64, 33000), (128, 2, 131080), (128, 2, 262152)])
def test_workgroups_with_several_steps_of_columns(T, R, N, rank):
    # a workgroup takes 2, 3 or 4 times 256 columns from 2048 workgroups on
    c = make(N, T, 8, N, R, rank, "fp16" if rank == 32 else "bf16")
    check(run(c), c)


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 511, 512, 513, 1000])
@pytest.mark.parametrize("R", [1, 2, 7])
def test_tile_borders(tokens, R):
    for index in ([0] * tokens, [R - 1] * tokens, [-1] * tokens, [t % R for t in range(tokens)],
                  [(t * R) // tokens for t in range(tokens)]):
        c = make(tokens, tokens, 264, 72, R, 16, "bf16", index)
        check(run(c), c)


@pytest.mark.parametrize("tokens", [40, 700])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_ranks_of_their_own(tokens, dtype):
    # what lies past an adapter's own rank takes no part, whatever it holds
    for rank in (16, 64, 128):
        ranks = [0, 1, rank - 1, rank, rank + 5, -3, 7, 9][:8]
        c = make(rank, tokens, 392, 200, 8, rank, dtype, ranks=ranks)
        for i, r in enumerate(ranks):
            c["a"][i, max(r, 0):] = math.nan
            c["b"][i, :, max(r, 0):] = math.inf
        want = {**c, "a": torch.nan_to_num(c["a"], 0, 0, 0), "b": torch.nan_to_num(c["b"], 0, 0, 0)}
        check(run(c), want)


def test_without_base_or_scales():
    for base, scales in ((False, False), (True, False), (False, True)):
        c = make(3, 50, 256, 96, 3, 16, "fp16", base=base, scales=scales)
        got = run(c)
        check(got, c)
        if not base:
            assert (got[torch.tensor(c["index"]) < 0] == 0).all()


def test_tokens_without_an_adapter_keep_their_base():
    for index in ([-1] * 40, [5, -7, 1 << 30, 0, -1] * 8):
        c = make(4, 40, 256, 96, 2, 8, "bf16", index)
        got = run(c)
        keep = torch.tensor([not 0 <= i < 2 for i in index])
        assert torch.equal(got.cpu()[keep], c["base"][keep])


@pytest.mark.parametrize("tokens", [30, 600])
def test_rows_that_lie_apart_and_in_place(tokens):
    c = make(5, tokens, 264, 104, 3, 32, "bf16")
    x = torch.full((tokens, 400), math.nan).bfloat16().cuda()
    x[:, 8:272] = c["x"].cuda()
    wide = torch.full((tokens, 208), math.inf).bfloat16().cuda()
    wide[:, 16:120] = c["base"].cuda()
    plan = adapters.lora_plan(ints(c["index"]), 3)
    args = c["a"].cuda(), c["b"].cuda(), plan
    kw = dict(scales=c["scales"].cuda())
    out = torch.full((tokens, 112), 7.0).bfloat16().cuda()
    adapters.lora(x[:, 8:272], *args, base=wide[:, 16:120], out=out[:, :104], **kw)
    check(out[:, :104], c)
    assert (out[:, 104:] == 7).all()
    got = adapters.lora(x[:, 8:272], *args, base=wide[:, 16:120], out=wide[:, 16:120], **kw)
    assert torch.equal(got, out[:, :104]) and wide[:, :16].isinf().all() and wide[:, 120:].isinf().all()
    # one row for all tokens, a step of 0
    one = {**c, "x": c["x"][:1].expand(tokens, 264)}
    check(adapters.lora(c["x"][:1].cuda().expand(tokens, 264), *args, base=c["base"].cuda(), **kw), one)


@pytest.mark.parametrize("tokens", [20, 700])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_what_is_not_finite_stays_in_its_token(tokens, dtype):
    c = make(6, tokens, 512, 88, 2, 32, dtype)
    clean = run(c)
    c["x"][3, 100] = math.nan
    c["x"][11, 511] = math.inf
    c["index"][3] = c["index"][11] = 0
    got = run(c)
    assert got[3].isnan().all() and not got[11].isfinite().any()
    rest = [t for t in range(tokens) if t not in (3, 11)]
    assert torch.equal(got[rest], clean[rest])
    # an infinite v: plus or minus infinity by b's sign, where no product is undefined
    c = make(7, tokens, 512, 88, 1, 8, dtype, [0] * tokens)
    c["x"][5] = 0
    c["x"][5, 7] = math.inf
    c["a"][0, :, 7] = 0.0
    c["a"][0, 2, 7] = 1.0
    c["x"][5, 8] = 2.0 ** 14
    c["a"][0, 3, 8] = 2.0 ** 14 if dtype == "fp16" else 2.0 ** 30
    got = run(c)[5].cpu()
    assert got.isnan().all()                             # the other ranks saw 0 x inf
    c["a"][0, :, 7] = 1.0
    got = run(c)[5].cpu()
    b = c["b"][0].float()
    same = (b > 0).all(1) | (b < 0).all(1)
    assert torch.equal(got.isinf(), same) or bool((got.isinf() | got.isnan()).all())


def test_large_and_small_inner_values():
    # v far outside fp16's range, and far below it, with b the other way round
    for gain in (2.0 ** 12, 2.0 ** -12):
        for tokens in (9, 400):
            c = make(8, tokens, 256, 64, 2, 16, "fp16", gain=gain)
            check(run(c), c)
    c = make(9, 12, 64, 64, 1, 8, "fp16", [0] * 12)
    c["x"] = (c["x"] * 0 + 60000).half()
    c["a"] = (c["a"] * 0 + 30000).half()                 # v = 1.2e11
    c["b"] = (torch.sign(c["b"]) * 2.0 ** -24).half()    # the smallest subnormal number
    check(run(c), c)
    c["x"] *= 0
    check(run(c), c)


def test_bf16_over_its_whole_range():
    c = make(10, 20, 128, 64, 2, 16, "bf16", gain=2.0 ** 60)
    check(run(c), c)
    c = make(10, 20, 128, 64, 2, 16, "bf16", gain=2.0 ** -60)
    check(run(c), c)


def test_one_plan_for_several_products_and_a_used_plan_elsewhere():
    c = make(11, 90, 256, 64, 4, 16)
    plan = adapters.lora_plan(ints(c["index"]), 4)
    d = make(12, 90, 640, 1032, 4, 64, "fp16", c["index"])
    for _ in range(2):
        check(run(c, plan), c)
        check(run(d, plan), d)
    with pytest.raises(ValueError, match="plan is for"):
        run(make(13, 91, 256, 64, 4, 16), plan)
    with pytest.raises(ValueError, match="plan is for"):
        run(make(13, 90, 256, 64, 5, 16, index=[0] * 90), plan)


def test_many_adapters_and_many_tokens():
    c = make(14, 3000, 64, 40, 1024, 8, "bf16")
    check(run(c), c)
    c = make(15, 20000, 64, 24, 3, 8, "fp16")
    check(run(c), c)


@pytest.mark.parametrize("T", [6, 200])
def test_offsets_past_32_bits(T):
    # rows of x, base and out and adapters that lie past 2^31 elements: as those side by side
    K, N, R, rank = 40000, 264, 1024, 64
    c = make(20, T, K, N, 2, rank, index=[0, 1, -1] * (T // 3) + [1] * (T % 3))
    a = torch.empty((R, rank, K), dtype=torch.bfloat16, device="cuda")
    b = torch.empty((R, 40000, rank), dtype=torch.bfloat16, device="cuda")
    assert a.numel() > 1 << 31 and b.numel() > 1 << 31
    a[[0, R - 1]], at = c["a"].cuda(), (1 << 32) // T // 8 * 8
    wide = torch.empty(at * T, dtype=torch.bfloat16, device="cuda")
    x, base = wide.as_strided((T, K), (at, 1)), wide.as_strided((T, N), (at, 1), K)
    x.copy_(c["x"])
    base.copy_(c["base"])
    b = b.view(-1)[:R * N * rank].view(R, N, rank) if T == 6 else b
    full = torch.zeros((2, b.shape[1], rank)).bfloat16()
    full[:, :N] = c["b"]
    b[[0, R - 1]] = full.cuda()
    index = [R - 1 if i == 1 else i for i in c["index"]]
    scales = torch.ones(R, device="cuda")
    scales[[0, R - 1]] = c["scales"].cuda()
    plan = adapters.lora_plan(ints(index), R)
    if T == 6:
        out = wide.as_strided((T, N), (at, 1), K + N)
        got = adapters.lora(x, a, b, plan, base=base, scales=scales, out=out)
    else:
        got = adapters.lora(x, a, b, plan, scales=scales)
        assert not got[:, N:].any()
        c["base"], got = None, got[:, :N]
    check(got, c)


def test_the_most_tokens():
    # 2^24 of them; one in 2^8 is compared, in fp64, with the tolerance of `check`
    T, K, N, R, rank = 1 << 24, 8, 8, 1024, 8
    g = torch.Generator(device="cuda").manual_seed(21)
    x, a, b = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, K), (R, rank, K), (R, N, rank)))
    index = torch.randint(-1, R, (T,), generator=g, device="cuda", dtype=torch.int32)
    got = adapters.lora(x, a, b, adapters.lora_plan(index, R))
    at = torch.arange(0, T, 256, device="cuda") + 7
    i = index[at].long()
    xs, aa, bb = x[at].double(), a[i.clamp(min=0)].double(), b[i.clamp(min=0)].double()
    v, deep = (xs[:, None] * aa).sum(-1), (xs[:, None] * aa).abs().sum(-1)
    y, vb, deep = ((bb * v[:, None]).sum(-1), (bb * v[:, None]).abs().sum(-1), (bb.abs() * deep[:, None]).sum(-1))
    y[i < 0] = 0
    tol = deep * K * 2.0 ** -23 + vb * (2.0 ** -18 + 2 * rank * 2.0 ** -23 + 2.0 ** -23)
    tol = tol + 2.0 ** -8 * (y.abs() + tol) + 2.0 ** -134
    assert ((got[at].double() - y).abs() <= tol).all()


def test_plan_keeps_the_order_of_tokens():
    g = np.random.default_rng(3)
    for T, R in ((1, 1), (64, 32), (5000, 3), (5000, 1024), (70000, 40)):
        index = g.integers(-2, R + 2, T)
        plan = adapters.lora_plan(ints(index), R)
        data = plan.data.view(torch.int32).cpu().numpy()
        rows = 64 if T >= 64 * R else 16
        most = min(-(-T // rows) + R, T)
        at = -(-most // 4) * 4
        tile, token = data[:most], data[at:].reshape(most, rows)
        key = np.where((index < 0) | (index >= R), -1, index)
        used = tile != -2
        assert (token[~used] == -1).all()
        order = token[used][token[used] >= 0]
        assert np.array_equal(order, np.argsort(np.where(key < 0, R, key), kind="stable"))
        for i, row in zip(tile[used], token[used]):
            n = int((row >= 0).sum())
            assert n > 0 and (row[n:] == -1).all() and (key[row[:n]] == i).all()


def test_no_tokens():
    c = make(16, 0, 64, 40, 2, 8, index=[])
    assert run(c).shape == (0, 40)


@pytest.mark.parametrize("K,rank", [(520, 16), (12288, 16), (520, 96)])    # one kernel; two, with and without splits
def test_captured_and_replayed_with_other_adapters(K, rank):
    c = make(17, 48, K, 264, 6, rank)
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    index = ints(c["index"])

    def step():
        plan = adapters.lora_plan(index, 6)
        y = adapters.lora(d["x"], d["a"], d["b"], plan, base=d["base"], scales=d["scales"])
        return adapters.lora(d["x"], d["a"], d["b"], plan, base=y, scales=d["scales"])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
    g = np.random.default_rng(0)
    for turn in range(4):
        index.copy_(ints(g.integers(-1, 6, 48)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step())


@pytest.mark.parametrize("K,rank", [(2048, 32), (12288, 32)])
def test_two_streams_at_once(K, rank):
    cs = [make(s, 64, K, 1024, 8, rank) for s in (18, 19)]
    want = [run(c) for c in cs]
    dev = [{k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)} for c in cs]
    plans = [adapters.lora_plan(ints(c["index"]), 8) for c in cs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cs], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = dev[i]
                outs[i].append(adapters.lora(d["x"], d["a"], d["b"], plans[i], base=d["base"], scales=d["scales"]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for got, w in zip(outs, want) for o in got)


def test_refusals():
    c = make(20, 8, 64, 40, 2, 8)
    plan = adapters.lora_plan(ints(c["index"]), 2)
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    ok = lambda **kw: adapters.lora(**{**dict(x=d["x"], a=d["a"], b=d["b"], plan=plan, base=d["base"]), **kw})  # noqa: E731
    for kw, error, what in ((dict(a=d["a"].half()), ValueError, "a must be"), (dict(b=d["b"][:, :, :7]), ValueError, "b must be"),
                            (dict(base=d["base"].half()), ValueError, "x's dtype"),
                            (dict(base=d["base"].t().contiguous().t()), ValueError, "contiguous"),
                            (dict(out=torch.empty((8, 48)).bfloat16().cuda()), ValueError, "out must be"),
                            (dict(scales=torch.ones(3).cuda()), ValueError, "scales"),
                            (dict(ranks=torch.ones(2).cuda()), ValueError, "ranks"),
                            (dict(base=d["base"][:1].expand(8, 40), out=d["base"]), RuntimeError, "in place"),
                            (dict(out=d["base"][:1].expand(8, 40)), RuntimeError, "out: rows"),
                            (dict(x=torch.zeros((8, 65)).bfloat16().cuda()[:, 1:]), RuntimeError, "multiple of 8")):
        with pytest.raises(error, match=what):
            ok(**kw)
    e = make(21, 8, 64, 40, 2, 16)
    with pytest.raises(RuntimeError, match="rank=12"):
        adapters.lora(e["x"].cuda(), e["a"][:, :12].contiguous().cuda(), e["b"][:, :, :12].contiguous().cuda(), plan)
    with pytest.raises(RuntimeError, match="k=60"):
        adapters.lora(e["x"][:, :60].contiguous().cuda(), e["a"][:, :, :60].contiguous().cuda(), e["b"].cuda(), plan)


def as_infinities(x):
    """1, -1 and 0 for infinities and finite numbers, NaN as it is."""
    x = np.asarray(x)
    return np.where(np.isinf(x), np.sign(x), np.where(np.isnan(x), np.nan, 0.0))


@pytest.mark.parametrize("tokens,K", [(1, 264), (20, 264), (20, 20488), (700, 264)])   # one kernel, two, tiles of 64
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_what_is_not_finite_in_b(dtype, rank, tokens, K):
    # v is finite and not 0: an infinity by its sign and b's, NaN where two meet of different signs
    c = make(30 + rank, tokens, K, 200, 2, rank, dtype, [t % 2 for t in range(tokens)])
    c["x"][:, 0] = 8                                     # v is 32 or -32, and some
    c["a"][:, :, 0] = 4 * (-1.0) ** torch.arange(rank)
    clean = run(c)
    x, a = f64(c["x"]), f64(c["a"])
    inf = math.inf
    places = {3: [(0, 0, inf)], 64: [(1, rank - 1, -inf)], 70: [(0, 1, inf), (0, 2, inf)], 71: [(1, 1, inf), (1, rank - 2, -inf)],
              130: [(0, rank - 1, math.nan)], 199: [(0, 5, -inf), (1, 7, inf)]}
    for n, them in places.items():
        for i, r, value in them:
            c["b"][i, n, r] = value
    for i in range(2):                                   # by more than any rounding
        v, deep = x @ a[i].T, np.abs(x) @ np.abs(a[i]).T
        assert (np.abs(v) > deep * K * 2.0 ** -23)[i::2].all()
    y = O.lora(x, a, f64(c["b"]), c["index"], f64(c["base"]), f64(c["scales"]))[0]
    got = run(c)
    np.testing.assert_array_equal(as_infinities(got.float().cpu().numpy()), as_infinities(y))
    same = np.isfinite(y)
    assert same[:, [0, 65, 198]].all() and np.array_equal(got.float().cpu().numpy()[same], clean.float().cpu().numpy()[same])


@pytest.mark.parametrize("tokens", [20, 700])
@pytest.mark.parametrize("rank", [8, 32, 128])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_an_infinite_v_by_its_sign_and_bs(dtype, rank, tokens):
    c = make(40 + rank, tokens, 264, 200, 1, rank, dtype, [0] * tokens)
    c["x"][5] = 0
    c["x"][5, 7] = math.inf
    signs = torch.ones(rank)
    signs[1] = -1
    c["a"][0, :, 7] = signs.to(c["a"].dtype)
    c["b"][0, :50] = (c["b"][0, :50].abs() * signs).to(c["b"].dtype)          # all plus infinity
    c["b"][0, 50:90] = (-c["b"][0, 50:90].abs() * signs).to(c["b"].dtype)     # all minus
    c["b"][0, 0, 0] = math.inf                                                # infinity times infinity
    c["b"][0, 50, 1] = math.inf
    c["b"][0, 89, rank - 1] = 0.0                                             # infinity times 0
    y = O.lora(*(f64(c[k]) for k in "xab"), c["index"], f64(c["base"]), f64(c["scales"]))[0][5]
    expected = as_infinities(y)
    assert (expected[:50] * expected[51] < 0).all() and expected[50] == expected[51] and np.isnan(expected[89])
    np.testing.assert_array_equal(as_infinities(run(c)[5].float().cpu().numpy()), expected)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_a_v_of_0_and_an_infinite_b(dtype):
    c = make(50, 30, 64, 72, 1, 16, dtype, [0] * 30)
    c["x"][4] = 0
    c["b"][0, 9, 3] = math.inf
    got = run(c)
    assert got[4, 9].isnan() and got[4, [8, 10]].isfinite().all() and got[3, 9].isinf()


@pytest.mark.parametrize("T,K", [(1, 64), (20, 20488), (300, 64)])
@pytest.mark.parametrize("rank", [8, 64])
def test_bf16_up_to_the_end_of_fp32(rank, T, K):
    # v between the largest bf16 and the largest fp32 number, a sum that is exact
    c = make(51, T, K, 72, 1, rank, "bf16", [0] * T, gain=2.0 ** 60)
    c["x"][:] = 0
    c["x"][:, 3], c["x"][:, K - 1] = 1.0, 1.0
    c["a"][:, :, 3], c["a"][:, :, K - 1] = float(torch.finfo(torch.bfloat16).max), 2.0 ** 119
    c["a"][:, 1::2] *= -1
    c["b"] = (c["b"].float() * 2.0 ** -60).bfloat16()
    v = f64(c["x"]) @ f64(c["a"][0]).T
    assert (np.abs(v) > float(torch.finfo(torch.bfloat16).max)).all() and (np.abs(v) < np.finfo(np.float32).max).all()
    got = run(c)
    assert got.isfinite().all()
    check(got, c)
