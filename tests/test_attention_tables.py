"""Block tables whose rows are not `pages` apart: what the binding hands to the
library must lead each sequence to its own row of the view (CPU), and attention
over such views equals attention over a plain copy (GPU)."""
import pytest
import torch

from weight_only_int4_unpack_amd import attn, serve_op
from weight_only_int4_unpack_amd import w4a16 as W

TABLE, STRIDE, SEQUENCES, PAGES = 12, 19, 20, 21     # fields of the packed arguments


class Here(torch.Tensor):
    """A CPU tensor that passes for one on a GPU: nothing is launched with it."""
    is_cuda = property(lambda self: True)


def here(x):
    return x.as_subclass(Here)


def views():
    """Name, table [B, pages] of int32."""
    flat = torch.arange(64, dtype=torch.int32)
    return [("plain", flat[:12].view(3, 4)), ("rows apart", flat.view(8, 8)[:3, :4]),
            ("expanded", flat[:4].view(1, 4).expand(8, 4)), ("one page, expanded", flat[:1].view(1, 1).expand(5, 1)),
            ("one row", flat.as_strided((1, 4), (1, 1)))]


def packed(monkeypatch, table, max_q=1):
    """Fields that tree_attention packs for `table`."""
    got = []
    monkeypatch.setattr(attn, "_call", lambda fn, dev, *a: got.append(attn._ATTEND.unpack(a[0])))
    monkeypatch.setattr(W, "_num_cus", lambda dev: 256)
    monkeypatch.setattr(W, "stream_workspace", lambda dev, n: None)
    B = table.shape[0]
    cache = attn.KVCache(*[torch.zeros((64, 1, 16, 64), dtype=torch.bfloat16) for _ in range(2)])
    attn.tree_attention(here(torch.zeros((B, 1, 64), dtype=torch.bfloat16)), cache, table,
                        torch.ones(B, dtype=torch.int32), torch.arange(B + 1, dtype=torch.int32), max_q)
    return got[0]


@pytest.mark.parametrize("name", [n for n, _ in views()])
def test_rows_that_are_handed_over_are_the_views_own(name, monkeypatch):
    table = dict(views())[name]
    f = packed(monkeypatch, table)
    assert f[SEQUENCES] == table.shape[0] and f[PAGES] == table.shape[1] and f[TABLE] == table.data_ptr()
    for b in range(table.shape[0]):
        assert f[TABLE] + 4 * b * f[STRIDE] == table[b].data_ptr()


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")
def test_the_library_takes_one_row_for_all_and_refuses_rows_that_overlap():
    P = 0x10000                              # aligned, never dereferenced on the host

    def status(stride):
        args = attn._ATTEND.pack(P, P, 0, 0, 4, 64, 8, 128, attn.KV_SAME, P, P, P, P, P, P, 0, 4, 1024, 128,
                                 stride, 2, 8, 2, 32, 0, 1, 0.1, 0)
        return W.lib().w4a16_tree_attention(args, P, 1 << 40, None)

    assert status(0) == status(8) == status(9) == W.ERR_DEVICE
    assert status(7) == status(1) == status(-1) == status(1 << 40) == W.ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("call", [attn.tree_attention, serve_op.tree_attention])
@pytest.mark.parametrize("news", [[1] * 8, [9] * 8])
def test_expanded_tables(news, call):
    # eight continuations of one prompt, on the prompt's pages
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = attn.KVCache(*[torch.randn((5, 2, 16, 64), generator=g, device="cuda").bfloat16() for _ in range(2)])
    q = torch.randn((sum(news), 4, 64), generator=g, device="cuda").bfloat16()
    row = torch.tensor([[3, 0, 4, 1]], dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, starts = ints([20 + 5 * b for b in range(8)]), ints([sum(news[:b]) for b in range(9)])
    want = call(q, cache, row.repeat(8, 1), lens, starts, max(news))
    got = call(q, cache, row.expand(8, 4), lens, starts, max(news))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(W.W4A16Error) as e:   # rows one into the other
        call(q, cache, torch.arange(16, dtype=torch.int32, device="cuda").as_strided((8, 4), (1, 1)), lens,
             starts, max(news))
    assert e.value.status == W.ERR_SHAPE
