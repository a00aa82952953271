"""GPU tests of the opaque operators around the weight products, and of the example
that runs them together."""
import importlib.util
import os
import sys

import pytest
import torch

from weight_only_int4_unpack_amd import attn, scoring, serve_op

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def problem(dtype=torch.float8_e4m3fn, T=6, H=8, G=2, D=64):
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    at = torch.arange(T, device="cuda")
    return dict(q=rand(T, H, D), k=rand(T, G, D), v=rand(T, G, D), slots=at + 16, pos=at,
                table=attn.rope_table(32, attn.rope_frequencies(32)),
                bt=torch.tensor([[1, 2], [1, 0]], dtype=torch.int32, device="cuda"),
                lens=torch.tensor([6, 2], dtype=torch.int32, device="cuda"),
                starts=torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda"),
                logits=rand(T, 1000), ids=at, cache=attn.kv_cache(4, G, D, 16, dtype))


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8, torch.bfloat16])
def test_operators_equal_the_bindings(dtype):
    p = problem(dtype)
    other = attn.kv_cache(4, 2, 64, 16, dtype)
    same = lambda a, b: torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
    assert same(serve_op.rope(p["q"], p["pos"], p["table"]), attn.rope(p["q"], p["pos"], p["table"]))
    q = serve_op.kv_write(p["k"], p["v"], p["slots"], p["cache"], p["pos"], p["table"], False, p["q"])
    q2 = attn.kv_write(p["k"], p["v"], p["slots"], other, p["pos"], p["table"], False, p["q"])
    assert same(q, q2)
    for a, b in zip(p["cache"], other):
        assert a is b is None or same(a, b)
    for a, b in zip(serve_op.kv_read(p["cache"], p["slots"]), attn.kv_read(other, p["slots"])):
        assert same(a, b)
    args = p["bt"], p["lens"], p["starts"], 4
    for a, b in zip(serve_op.tree_attention(q, p["cache"], *args),
                    attn.tree_attention(q, other, *args)):
        assert same(a, b)
    for a, b in zip(serve_op.token_logprobs(p["logits"], p["ids"], 9),
                    scoring.token_logprobs(p["logits"], p["ids"], 9)):
        assert same(a, b)


def test_opcheck():
    p = problem(torch.int8)             # the check scales its inputs, which torch does not for fp8
    ops = torch.ops.w4a16
    cases = [
        (ops.rope, (p["q"], p["pos"], p["table"], False, False)),
        (ops.kv_write, (p["k"], p["v"], p["slots"], *p["cache"], p["pos"], p["table"], False, p["q"])),
        (ops.kv_write, (p["k"], p["v"], p["slots"], *p["cache"])),
        (ops.kv_read, (*p["cache"], p["slots"], torch.bfloat16)),
        (ops.tree_attention, (p["q"], *p["cache"], p["bt"], p["lens"], p["starts"], 4, None, 0.125)),
        (ops.token_logprobs, (p["logits"], p["ids"], 4)),
    ]
    for op, args in cases:
        torch.library.opcheck(op.default, args, test_utils=("test_schema", "test_faketensor"))


def test_a_compiled_step_equals_the_eager_one():
    def step(q, k, v, slots, cache, pos, table, bt, lens, starts):
        q = serve_op.kv_write(k, v, slots, cache, pos, table, False, q)
        return serve_op.tree_attention(q, cache, bt, lens, starts, 4)[0]
    names = ("q", "k", "v", "slots", "cache", "pos", "table", "bt", "lens", "starts")
    a, b = problem(), problem()
    want = step(*(a[n] for n in names))
    got = torch.compile(step, backend="aot_eager", fullgraph=True)(*(b[n] for n in names))
    assert torch.equal(got, want)
    for x, y in zip(a["cache"], b["cache"]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def example():
    spec = importlib.util.spec_from_file_location("verify_tree",
                                                  os.path.join(ROOT, "examples", "verify_tree.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["verify_tree"] = m
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ["e4m3", "int8", "16"])
def test_example_accepts_what_single_tokens_give(cache):
    # A tree and single tokens run different kernels (row counts, splits), so logits
    # agree to bf16 steps and a choice between near-equals may differ: the texts are
    # compared up to there, by scoring the drafted run's text in one pass. Its chosen
    # tokens are the pass's best or behind it by the noise of two bf16 logits and of
    # the layers under them. Each layer adds at most two bf16 steps to a normalised
    # state, so of logits of unit gain (standard deviation 1, below 6) with 2 layers
    # 2 * (2 + 1) * 6 * 2^-8 < 0.15. A moved key of an 8-bit cache is read and stored
    # again: a half-step of bf16 and then the same code, or the next (e4m3 steps of
    # 2^-3 in a state made of many keys): 0.3.
    m = example()
    s = m.Sizes()
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (33, 1, 20)]
    model = m.Decoder(s, 3, m.CACHES[cache])
    texts, scores = m.generate(model, prompts, 6)
    assert all(len(t) >= len(p) + 6 for t, p in zip(texts, prompts))
    fresh = m.Decoder(s, 3, m.CACHES[cache])
    starts, _, top, _ = m.run(fresh, texts, [0] * 3, [m.chain(t) for t in texts])
    for b, (t, p) in enumerate(zip(texts, prompts)):
        first = starts[b] + len(p) - 1
        best = top[first:starts[b + 1] - 1, 0].tolist()
        assert len(best) == len(scores[b])
        assert max(abs(x - y) for x, y in zip(best, scores[b])) < (0.15 if cache == "16" else 0.3)


def test_example_runs():
    example().main(["--steps", "3"])
