"""CPU tests of the opaque operators around the weight products (no kernel runs):
fake implementations report shapes, dtypes and devices, a traced graph keeps
each as one call node, only ``kv_write`` writes inputs, malformed calls fail."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

from weight_only_int4_unpack_amd import attn, serve_op

I32, I64, F32 = torch.int32, torch.int64, torch.float32


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, device="cuda", dtype=dtype)


def inputs(dtype=torch.float8_e4m3fn, T=6, B=2, H=8, G=2, D=64):
    c = attn.kv_cache(5, G, D, 16, dtype, "cuda")
    return dict(q=empty(T, H, D), k=empty(T, G, D), v=empty(T, G, D), cache=c,
                slots=empty(T, dtype=I64), pos=empty(T, dtype=I64), table=empty(100, 32, dtype=F32),
                bt=empty(B, 4, dtype=I32), lens=empty(B, dtype=I32), starts=empty(B + 1, dtype=I32),
                mask=empty(T, 1, dtype=I64), logits=empty(T, 1000), ids=empty(T, dtype=I64))


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8, torch.bfloat16])
def test_fakes_report_shapes(dtype):
    with FakeTensorMode():
        i = inputs(dtype)
        out = serve_op.rope(i["q"], i["pos"], i["table"])
        assert out.shape == i["q"].shape and out.dtype == torch.bfloat16
        q = serve_op.kv_write(i["k"], i["v"], i["slots"], i["cache"], i["pos"], i["table"], False, i["q"])
        assert q.shape == i["q"].shape and q.is_contiguous() and q.device == i["q"].device
        assert serve_op.kv_write(i["k"], i["v"], i["slots"], i["cache"]) is None
        for x in serve_op.kv_read(i["cache"], i["slots"]):
            assert x.shape == i["k"].shape and x.dtype == torch.bfloat16
        o, lse = serve_op.tree_attention(q, i["cache"], i["bt"], i["lens"], i["starts"], 4, i["mask"])
        assert o.shape == q.shape and lse.shape == q.shape[:2] and lse.dtype == F32
        lp, ent, top, at = serve_op.token_logprobs(i["logits"], i["ids"], 7)
        assert lp.shape == ent.shape == (6,) and top.shape == at.shape == (6, 7)
        assert top.dtype == F32 and at.dtype == I64


def test_a_graph_keeps_one_node_each():
    def step(q, k, v, slots, kc, vc, ks, vs, pos, table, bt, lens, starts, logits, ids):
        cache = attn.KVCache(kc, vc, ks, vs)
        q = serve_op.kv_write(k, v, slots, cache, pos, table, False, q)
        o, _ = serve_op.tree_attention(q, cache, bt, lens, starts, 4)
        return o, serve_op.token_logprobs(logits, ids, 3)[0]
    with FakeTensorMode():
        i = inputs()
        args = [i[n] for n in ("q", "k", "v", "slots")] + list(i["cache"]) + \
               [i[n] for n in ("pos", "table", "bt", "lens", "starts", "logits", "ids")]
        gm = make_fx(step)(*args)
    calls = [n.target for n in gm.graph.nodes
             if n.op == "call_function" and "w4a16" in str(n.target)]
    ops = torch.ops.w4a16
    assert calls == [ops.kv_write.default, ops.tree_attention.default, ops.token_logprobs.default]


def test_only_the_cache_is_written():
    ops = torch.ops.w4a16
    for op in (ops.rope, ops.kv_read, ops.tree_attention, ops.token_logprobs):
        assert not op.default._schema.is_mutable
    written = [a.name for a in ops.kv_write.default._schema.arguments
               if a.alias_info is not None and a.alias_info.is_write]
    assert written == ["k_cache", "v_cache", "k_scale", "v_scale"]


@pytest.mark.parametrize("bad", ["positions", "table", "slots", "heads", "scales", "dtype", "q alone",
                                 "lens", "starts", "mask", "ids", "top_k", "read dtype"])
def test_fakes_refuse_malformed_calls(bad):
    with FakeTensorMode():
        i = inputs()
        def write(**k):
            j = {**i, **k}
            serve_op.kv_write(j["k"], j["v"], j["slots"], j["cache"], j["pos"], j["table"], False, j["q"])
        def attend(**k):
            j = {**i, **k}
            serve_op.tree_attention(j["q"], j["cache"], j["bt"], j["lens"], j["starts"], 4, j["mask"])
        calls = {
            "positions": lambda: serve_op.rope(i["q"], empty(5, dtype=I64), i["table"]),
            "table": lambda: serve_op.rope(i["q"], i["pos"], empty(9, 66, dtype=F32)),
            "slots": lambda: write(slots=empty(6, dtype=I32)),
            "heads": lambda: write(k=empty(6, 3, 64), v=empty(6, 3, 64)),
            "scales": lambda: write(cache=i["cache"]._replace(v_scale=None)),
            "dtype": lambda: attend(cache=attn.kv_cache(5, 2, 64, 16, torch.float16, "cuda")),
            "q alone": lambda: write(pos=None, table=None),
            "lens": lambda: attend(lens=empty(3, dtype=I32)),
            "starts": lambda: attend(starts=empty(2, dtype=I32)),
            "mask": lambda: attend(mask=empty(5, 1, dtype=I64)),
            "ids": lambda: serve_op.token_logprobs(i["logits"], empty(5, dtype=I64)),
            "top_k": lambda: serve_op.token_logprobs(i["logits"], i["ids"], 65),
            "read dtype": lambda: serve_op.kv_read(i["cache"], i["slots"], F32),
        }
        with pytest.raises(Exception, match="must|needs|are needed"):
            calls[bad]()
