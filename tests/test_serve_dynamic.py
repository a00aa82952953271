"""The opaque operators around the weight products under dynamic shapes: one graph
holds for any number of tokens, sequences and pages."""
import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

from weight_only_int4_unpack_amd import attn, serve_op


def inputs(tokens, sequences, pages, device, dtype=torch.int8, top=100):
    g = torch.Generator().manual_seed(tokens)
    rand = lambda *s: torch.randn(s, generator=g).bfloat16().to(device)      # noqa: E731
    k, v = torch.zeros((2, pages, 2, 16, 64), dtype=dtype, device=device)
    ks, vs = torch.zeros((2, pages, 2, 16), device=device)
    each = tokens // sequences
    return [rand(tokens, 8, 64), rand(tokens, 2, 64), rand(tokens, 2, 64),
            torch.arange(tokens, device=device), k, v, ks, vs, torch.rand((top, 32), generator=g).to(device),
            torch.arange(sequences * 4, dtype=torch.int32).view(sequences, 4).to(device) % pages,
            torch.full((sequences,), 60, dtype=torch.int32, device=device),
            (torch.arange(sequences + 1, dtype=torch.int32) * each).to(device), rand(tokens, 1000)]


def step(q, k, v, at, kc, vc, ks, vs, table, pages, lens, starts, logits):
    cache = attn.KVCache(kc, vc, ks, vs)
    q = serve_op.kv_write(serve_op.rope(k, at, table), v, at, cache, at, table, False, q)
    out, lse = serve_op.tree_attention(q, cache, pages, lens, starts, 64)
    back = serve_op.kv_read(cache, at, torch.bfloat16)
    return out, lse, *back, *serve_op.token_logprobs(logits, at, 3)


def test_a_traced_graph_keeps_its_sizes_free():
    gm = make_fx(step, tracing_mode="symbolic")(*inputs(12, 3, 7, "cpu"))
    shapes = [n.meta["val"].shape for n in gm.graph.nodes if n.op == "placeholder"]
    assert not isinstance(shapes[0][0], int) and not isinstance(shapes[4][0], int)      # tokens, pages
    calls = [str(n.target) for n in gm.graph.nodes if n.op == "call_function" and "w4a16" in str(n.target)]
    assert calls == [f"w4a16.{n}.default" for n in ("rope", "kv_write", "tree_attention", "kv_read", "token_logprobs")]
    out = next(n for n in gm.graph.nodes if n.op == "output").args[0]
    assert out[0].meta["val"].shape[0] == shapes[0][0] and not isinstance(out[0].meta["val"].shape[0], int)


@pytest.mark.gpu
def test_one_compiled_step_for_several_sizes():
    compiled = torch.compile(step, backend="aot_eager", fullgraph=True, dynamic=True)
    for tokens, sequences, pages in ((12, 3, 7), (40, 4, 9), (7, 7, 30)):
        a, b = inputs(tokens, sequences, pages, "cuda"), inputs(tokens, sequences, pages, "cuda")
        want, got = step(*a), compiled(*b)
        for x, y in zip([*want, *a[4:8]], [*got, *b[4:8]]):
            assert torch.equal(x, y)
