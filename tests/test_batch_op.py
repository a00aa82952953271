"""CPU tests of verification, pages and adapters as opaque operators (no kernel runs):
fake implementations report shapes, dtypes and devices, a traced graph keeps each as one
call node and its sizes free, schemas say what is written, malformed calls fail."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

from weight_only_int4_unpack_amd import adapters, attn, batch_op, paging

I32, I64, F32, U8 = torch.int32, torch.int64, torch.float32, torch.uint8
OPS = torch.ops.w4a16


def empty(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.empty(shape, device=device, dtype=dtype)


def group(dtype=torch.int8, n=2, device="cuda"):
    return paging.CacheGroup(tuple(attn.kv_cache(9, 2, 64, 16, dtype, device) for _ in range(n)), None)


def pool(device="cuda"):
    return paging.page_pool(9, 3, 4, 16, device)


def verify(T=6, B=2, V=1000, **kw):
    a = dict(logits=empty(T, V), ids=empty(T, dtype=I64), q_starts=empty(B + 1, dtype=I32), max_q=4,
             uniforms=empty(T, dtype=F32), final_uniforms=empty(B, dtype=F32), parents=empty(T, dtype=I32),
             draft_probs=None, temperatures=empty(B, dtype=F32))
    return batch_op.verify_drafts(**{**a, **kw})


def lora(T=6, K=64, N=72, R=3, rank=8, **kw):
    a = dict(x=empty(T, K), a=empty(R, rank, K), b=empty(R, N, rank),
             plan=batch_op.lora_plan(empty(T, dtype=I32), R), base=empty(T, N), scales=empty(R, dtype=F32),
             ranks=empty(R, dtype=I32))
    return batch_op.lora(**{**a, **kw})


def compact(g=None, B=2, **kw):
    a = dict(block_table=empty(B, 4, dtype=I32), kv_lens=empty(B, dtype=I32), q_starts=empty(B + 1, dtype=I32),
             path=empty(B, 4, dtype=I32), counts=empty(B, dtype=I32))
    return batch_op.kv_compact(g or group(), **{**a, **kw})


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8, torch.bfloat16])
def test_fakes_report_shapes(dtype):
    with FakeTensorMode():
        tokens, path, counts = verify()
        assert tokens.shape == path.shape == (2, 4) and counts.shape == (2,)
        assert tokens.dtype == I64 and path.dtype == counts.dtype == I32
        for change in (batch_op.pages_resize, batch_op.pages_fork):
            for x in change(pool(), empty(2, dtype=I32), empty(2, dtype=I32)):
                assert x.shape == (2,) and x.dtype == I32
        assert batch_op.kv_copy_pages(group(dtype), empty(2, dtype=I32), empty(2, dtype=I32)) is None
        assert compact(group(dtype)).shape == (2,)
        y = lora()
        assert y.shape == (6, 72) and y.dtype == torch.bfloat16 and y.is_contiguous()


def test_a_plan_of_either_tile_size_fits():
    for tokens in (0, 1, 15, 16, 17, 63, 64, 65, 100, 127, 128, 1000, 4095, 4096, 65536, 65537, 1 << 24):
        for n in (1, 2, 3, 15, 16, 63, 64, 65, 255, 1023, 1024):
            assert adapters.plan_bytes(tokens, n) <= batch_op._plan_room(tokens, n)


def test_schemas_say_what_is_written():
    wrote = lambda op: [a.name for a in op.default._schema.arguments                                   # noqa: E731
                        if a.alias_info is not None and a.alias_info.is_write]
    assert wrote(OPS.pages_resize) == wrote(OPS.pages_fork) == ["refs", "block_table", "pool_lens"]
    assert wrote(OPS.kv_copy_pages) == wrote(OPS.kv_compact) == ["k", "v", "k_scales", "v_scales"]
    for op in (OPS.verify_drafts, OPS.lora_plan, OPS.lora):
        assert not op.default._schema.is_mutable


def step(logits, ids, starts, uniforms, finals, parents, refs, table, lens, k, v, ks, vs, rows, x, a, b, index):
    # sequences `rows` verify and compact, give pages back and go on as the rows behind them too
    B = rows.shape[0]
    p = paging.PagePool(refs, table, lens, 16)
    g = paging.CacheGroup((attn.KVCache(k, v, ks, vs),), None)
    y = batch_op.lora(x, a, b, batch_op.lora_plan(index, a.shape[0]))
    tokens, path, counts = batch_op.verify_drafts(logits, ids, starts, 8, uniforms, finals, parents)
    new = batch_op.kv_compact(g, table[:B], lens[:B].clone(), starts, path, counts)
    served, src, dst = batch_op.pages_resize(p, rows, new)
    batch_op.kv_copy_pages(g, src, dst)
    forked, src, dst = batch_op.pages_fork(p, rows, rows + B)
    batch_op.kv_copy_pages(g, src, dst)
    return y, tokens, path, counts, new, served, forked


def sizes(T, B, device, seed=0, R=3, vocab=500):
    """Inputs of a step: B sequences of ragged trees, T nodes, with pages for what they hold."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s, dtype=F32: torch.rand(s, generator=g).to(dtype).to(device)                       # noqa: E731
    ints = lambda x, dtype=I32: torch.tensor(x, dtype=dtype, device=device)                            # noqa: E731
    cuts = [T * i // B for i in range(B + 1)]
    held = [int(n) + hi - lo for n, lo, hi in
            zip(torch.randint(0, 50 - T // B, (B,), generator=g), cuts, cuts[1:])]
    parents = [j - 1 if j < 2 else int(torch.randint(0, j, (), generator=g)) for lo, hi in zip(cuts, cuts[1:])
               for j in range(hi - lo)]
    pages = 10 * B
    order = torch.randperm(pages, generator=g).tolist()
    table, refs = [[-1] * 5 for _ in range(2 * B)], [0] * pages
    for b in range(B):
        for j in range(-(-held[b] // 16)):
            table[b][j] = order.pop()
            refs[table[b][j]] = 1
    codes = torch.randint(-127, 128, (2, pages, 2, 16, 64), generator=g).to(torch.int8).to(device)
    return [rand(T, vocab) * 3, torch.randint(0, vocab, (T,), generator=g).to(device), ints(cuts), rand(T) * 0.01, rand(B),
            ints(parents), ints(refs), ints(table), ints(held + [0] * B), codes[0].clone(), codes[1].clone(),
            rand(pages, 2, 16), rand(pages, 2, 16), torch.arange(B, dtype=I32, device=device),
            rand(T, 64, dtype=torch.bfloat16), rand(R, 8, 64, dtype=torch.bfloat16),
            rand(R, 72, 8, dtype=torch.bfloat16), torch.randint(-1, R, (T,), generator=g).int().to(device)]


def test_a_traced_graph_keeps_one_node_each_and_its_sizes_free():
    gm = make_fx(step, tracing_mode="symbolic")(*sizes(12, 5, "cpu"))
    shapes = [n.meta["val"].shape for n in gm.graph.nodes if n.op == "placeholder"]
    assert not isinstance(shapes[0][0], int) and not isinstance(shapes[6][0], int)      # tokens, pages
    calls = [str(n.target) for n in gm.graph.nodes if n.op == "call_function" and "w4a16" in str(n.target)]
    assert calls == [f"w4a16.{n}.default" for n in ("lora_plan", "lora", "verify_drafts", "kv_compact",
                                                    "pages_resize", "kv_copy_pages", "pages_fork", "kv_copy_pages")]
    out = next(n for n in gm.graph.nodes if n.op == "output").args[0]
    assert out[0].meta["val"].shape[0] == shapes[0][0] and not isinstance(out[0].meta["val"].shape[0], int)


@pytest.mark.parametrize("call", [
    lambda: verify(ids=empty(5, dtype=I64)), lambda: verify(logits=empty(6, 9, dtype=I32)),
    lambda: verify(q_starts=empty(3, dtype=I64)), lambda: verify(uniforms=empty(6)),
    lambda: verify(final_uniforms=empty(3, dtype=F32)), lambda: verify(parents=empty(6, dtype=I64)),
    lambda: verify(draft_probs=empty(6, 1000, dtype=F32)),
    lambda: verify(parents=None, draft_probs=empty(6, 999, dtype=F32)), lambda: verify(temperatures=empty(1, dtype=F32)),
    lambda: batch_op.pages_resize(pool(), empty(2, dtype=I64), empty(2, dtype=I32)),
    lambda: batch_op.pages_resize(pool(), empty(2, dtype=I32), empty(3, dtype=I32)),
    lambda: batch_op.pages_fork(pool()._replace(lens=empty(2, dtype=I32)), empty(2, dtype=I32), empty(2, dtype=I32)),
    lambda: batch_op.kv_copy_pages(group(), empty(2, dtype=I32), empty(2, dtype=I64)),
    lambda: batch_op.kv_copy_pages(paging.CacheGroup((*group(n=1).caches, attn.kv_cache(8, 2, 64, 16, torch.int8, "cuda")),
                                                     None), empty(2, dtype=I32), empty(2, dtype=I32)),
    lambda: compact(path=empty(2, 4, dtype=I64)), lambda: compact(counts=empty(3, dtype=I32)),
    lambda: compact(q_starts=empty(2, dtype=I32)), lambda: compact(block_table=empty(2, 4, dtype=I64)),
    lambda: batch_op.lora_plan(empty(6, dtype=I64), 3), lambda: lora(x=empty(6, 64, dtype=F32)),
    lambda: lora(a=empty(3, 8, 72)), lambda: lora(b=empty(2, 72, 8)), lambda: lora(base=empty(6, 64)),
    lambda: lora(scales=empty(2, dtype=F32)), lambda: lora(ranks=empty(3, dtype=I64)),
    lambda: lora(plan=adapters.LoraPlan(empty(900, dtype=U8), 6, 4)),
    lambda: lora(plan=adapters.LoraPlan(empty(900, dtype=I32), 6, 3)),
])
def test_fakes_refuse_malformed_calls(call):
    with FakeTensorMode(), pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("made_for,rows", [(200, 6), (2, 64), (7, 6), (5, 6), (65, 64)])
def test_a_plan_of_another_step_is_refused(made_for, rows):
    # 64 rows and 2, or 200 and 6, have plans whose memory is large enough for each other
    with FakeTensorMode():
        plan = batch_op.lora_plan(empty(made_for, dtype=I32), 3)
        with pytest.raises(ValueError, match=f"{made_for} tokens and 3 adapters, not {rows} and 3"):
            lora(T=rows, plan=plan)
        with pytest.raises(ValueError, match="the plan is for"):
            lora(T=made_for, R=4, plan=plan)
        assert lora(T=made_for, plan=plan).shape == (made_for, 72)


def test_a_traced_graph_ties_the_plan_to_the_rows():
    def product(x, a, b, index):
        return batch_op.lora(x, a, b, batch_op.lora_plan(index, a.shape[0]))
    args = [torch.zeros(s).bfloat16() for s in ((12, 64), (3, 8, 64), (3, 72, 8))]
    gm = make_fx(product, tracing_mode="symbolic")(*args, torch.zeros(12, dtype=I32))
    rows = next(n for n in gm.graph.nodes if n.op == "placeholder").meta["val"].shape[0]
    assert not isinstance(rows, int)
    with pytest.raises(ValueError, match="the plan is for"):
        make_fx(product, tracing_mode="symbolic")(*args, torch.zeros(11, dtype=I32))
