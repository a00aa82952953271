"""GPU tests of verification, pages and adapters together: as torch operators, compiled,
captured into a graph, and as the example runs them over a whole generation."""
import pytest
import torch
from test_batch_op import sizes, step
from test_gpu_serve_op import example

from weight_only_int4_unpack_amd import adapters, attn, batch_op, paging, scoring

pytestmark = pytest.mark.gpu
CASES = [(12, 5), (40, 5), (7, 7), (96, 12), (3, 1)]


def same(a, b):
    return all(torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8)) for x, y in zip(a, b, strict=True))


def bindings(logits, ids, starts, uniforms, finals, parents, refs, table, lens, k, v, ks, vs, rows, x, a, b, index):
    """test_batch_op.step by the bindings."""
    B = rows.shape[0]
    p, g = paging.PagePool(refs, table, lens, 16), paging.cache_group([attn.KVCache(k, v, ks, vs)])
    y = adapters.lora(x, a, b, adapters.lora_plan(index, a.shape[0]))
    tokens, path, counts = scoring.verify_drafts(logits, ids, starts, 8, uniforms, finals, parents)
    new = paging.kv_compact(g, table[:B], lens[:B].clone(), starts, path, counts)
    served, src, dst = paging.pages_resize(p, rows, new)
    paging.kv_copy_pages(g, src, dst)
    forked, src, dst = paging.pages_fork(p, rows, rows + B)
    paging.kv_copy_pages(g, src, dst)
    return y, tokens, path, counts, new, served, forked


@pytest.mark.parametrize("T,B", CASES)
def test_operators_equal_the_bindings(T, B):
    a, b = sizes(T, B, "cuda", T), sizes(T, B, "cuda", T)
    got = step(*a)
    assert same(got, bindings(*b)) and same(a, b)
    assert got[5].all() and got[6].all() and (got[4] > 0).all()
    # what sequences hold and how often each page is held
    refs, table, lens = (t.cpu() for t in a[6:9])
    count = torch.zeros_like(refs)
    for row, n in zip(table.tolist(), lens.tolist()):
        for page in row[:-(-n // 16)]:
            count[page] += 1
    assert torch.equal(count, refs)


def test_opcheck():
    a = sizes(40, 5, "cuda")
    ops, utils = torch.ops.w4a16, ("test_schema", "test_faketensor")
    lists = [a[9]], [a[10]], [a[11]], [a[12]]
    rows, x, la, lb, index = a[13:]
    pages = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    plan = ops.lora_plan(index, 3)
    for op, args in [
            (ops.verify_drafts, (*a[:3], 8, *a[3:6], None, None)),
            (ops.verify_drafts, (*a[:3], 8, *a[3:5], None, a[0].softmax(-1), torch.ones(5, device="cuda"))),
            (ops.pages_resize, (*a[6:9], 16, rows, rows)), (ops.pages_fork, (*a[6:9], 16, rows, rows + 5)),
            (ops.kv_copy_pages, (*lists, pages, pages + 2)),
            (ops.kv_copy_pages, (*([c[0].half()] for c in lists[:2]), [], [], pages, pages + 2)),
            (ops.lora_plan, (index, 3)), (ops.lora, (x, la, lb, plan, None, None, None))]:
        torch.library.opcheck(op.default, args, test_utils=utils)
    tokens, path, counts = ops.verify_drafts(*a[:3], 8, *a[3:6])
    torch.library.opcheck(ops.kv_compact.default, (*lists, a[7][:5], a[8][:5], a[2], path, counts), test_utils=utils)


def test_one_compiled_step_for_several_sizes():
    compiled = torch.compile(step, backend="aot_eager", fullgraph=True, dynamic=True)
    for T, B in CASES:
        a, b = sizes(T, B, "cuda", T), sizes(T, B, "cuda", T)
        assert same(bindings(*a), compiled(*b)) and same(a, b)


def test_a_captured_step_replayed():
    a = sizes(40, 5, "cuda", 1)
    names = len(a)
    bindings(*[t.clone() for t in a])                         # what a first call makes is there
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        out = bindings(*a)
    torch.cuda.current_stream().wait_stream(s)
    for seed in (2, 1, 3, 4):
        other = sizes(40, 5, "cuda", seed)
        for i in range(names):
            a[i].copy_(other[i])
        graph.replay()
        torch.cuda.synchronize()
        assert same(bindings(*other), out) and same(a, other)  # eager work between the replays


# A text that drafts, forks and compaction made is scored again by a fresh model in one pass,
# which shares no pages, compacts nothing and gives each sequence its adapter alone. The two
# passes run different kernels; each layer adds at most three bf16 steps to a normalised state
# (the product, the adapter's sum, the output), so two logits of unit gain (standard deviation
# 1, below 6) with 2 layers and the head differ by less than 2 (3 * 2 / 2 + 1) 6 2^-8 < 0.19,
# and so do log probabilities, whose normaliser moves by no more than the logits do: 0.38.
# An 8-bit cache may store the next code for a state between two (e4m3 steps of 2^-3 in a
# state made of many keys): 0.15 more.
@pytest.mark.parametrize("temperature", [0.0, 0.8])
@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_a_generation_equals_its_text_scored_alone(cache, temperature):
    m = example()
    s = m.Sizes()
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (33, 1, 20, 16)]
    P, rows = len(prompts), 3 * len(prompts)
    model = m.Decoder(s, rows, m.CACHES[cache], adapters=2)
    texts, scores = m.generate(model, prompts, 6, samples=3, temperature=temperature)
    assert all(len(t) >= len(prompts[b % P]) + 6 for b, t in enumerate(texts))
    fresh = m.Decoder(s, rows, m.CACHES[cache], adapters=2)
    fresh.adapter = torch.arange(rows, dtype=torch.int32, device="cuda") % P % 3    # a prompt's, for all its samples
    p = m.forward(fresh, [0] * rows, [m.chain(t) for t in texts])
    chosen = torch.cat([p.tokens[1:], p.tokens[:1]])          # the token after each; the last ones' are not used
    logprob, _, top, _ = scoring.token_logprobs(p.logits, chosen, 1)
    bound = 0.38 if cache == "16" else 0.53
    for b, t in enumerate(texts):
        own = len(prompts[b % P])
        at = slice(p.starts[b] + own - 1, p.starts[b + 1] - 1)
        assert len(scores[b]) == len(t) - own
        alone = logprob[at].tolist()
        assert max(abs(x - y) for x, y in zip(alone, scores[b], strict=True)) < bound
        if temperature == 0:
            assert (top[at, 0] - logprob[at]).max() < bound   # its choices, or as good as they
    model.resize(torch.zeros(rows, dtype=torch.int32, device="cuda"))
    assert not model.pool.refs.any() and (model.pool.block_table == -1).all()


def test_example_with_all_options_runs():
    example().main(["--steps", "3", "--adapters", "2", "--samples", "2", "--temperature", "0.7"])


@pytest.mark.parametrize("made_for,rows", [(200, 6), (2, 64)])
def test_a_plan_of_another_step_is_refused(made_for, rows):
    x, la, lb, index = sizes(rows, 2, "cuda")[14:]
    plan = batch_op.lora_plan(torch.zeros(made_for, dtype=torch.int32, device="cuda"), 3)
    for lora in (batch_op.lora, adapters.lora):
        with pytest.raises(ValueError, match="the plan is for"):
            lora(x, la, lb, plan)
    assert torch.equal(batch_op.lora(x, la, lb, batch_op.lora_plan(index, 3)),
                       adapters.lora(x, la, lb, adapters.lora_plan(index, 3)))


@pytest.mark.parametrize("prompt,steps", [(20, 30), (40, 1)])
def test_a_text_that_does_not_fit_stops_the_example(prompt, steps):
    # two pages a sequence: the text grows past them, or never fits
    m = example()
    s = m.Sizes(pages_each=2)
    model = m.Decoder(s, 2, None)
    with pytest.raises(RuntimeError, match=r"no room for sequences \[0\]: up to 32 tokens each"):
        m.generate(model, [list(range(prompt)), [1]], steps, drafts=False)


def test_a_fork_without_free_pages_stops_the_example():
    m = example()
    model = m.Decoder(m.Sizes(pages_each=2), 4, None)
    model.resize(m.ints([20, 32, 0, 0], torch.int32))
    model.pool.refs[model.pool.refs == 0] = 1                 # others hold the rest
    with pytest.raises(RuntimeError, match=r"no room for sequences \[2\]: .* 0 pages free"):
        model.fork([0, 1], [2, 3])
    assert model.pool.lens.tolist() == [20, 32, 0, 32]        # full pages alone are shared
