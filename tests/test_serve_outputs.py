"""Outputs whose heads lie one in another are refused: several lanes would write one
place, and a rotation in place would read what another has written."""
import pytest
import torch

from weight_only_int4_unpack_amd import attn
from weight_only_int4_unpack_amd import w4a16 as W

P = 0x10000                       # aligned, never dereferenced on the host

# tokens, heads, token stride, head stride of [tokens, heads, 64]
OVERLAPPING = [(4, 8, 0, 64), (4, 8, 512, 0), (4, 8, 0, 0), (4, 8, 448, 64), (4, 8, 64, 192), (2, 2, 56, 512),
               (2, 2, 512, 56), (1, 2, 512, 32), (2, 1, 32, 512), (2, 1 << 28, 1 << 33, 64)]
APART = [(4, 8, 512, 64), (4, 8, 64, 256), (4, 8, 1024, 128), (4, 8, 64, 1 << 39), (1, 8, 0, 64), (4, 1, 64, 0),
         (1, 1, 0, 0), (2, 1 << 28, 1 << 34, 64)]


def _rope(T, H, ot, oh, in_place=False):
    xt, xh = (ot, oh) if in_place else (64 * H if T > 1 else 0, 64 if H > 1 else 0)
    return W.lib().w4a16_rope(attn._ROPE.pack(P, P if in_place else 2 * P, P, P, T, xt, xh, ot, oh, 32, H, 64, 64,
                                              0, 0, 1), None)


def _write(T, H, ot, oh):
    return W.lib().w4a16_kv_write(attn._WRITE.pack(P, P, P, P, 4, 64, 8, 64, attn.KV_E4M3, P, P, P, P, 2 * P, P, P,
                                                   T, 512, 64, 512, 64, 64 * H if T > 1 else 0, 64, ot, oh, 32, H, 64,
                                                   0, 1), None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")
@pytest.mark.parametrize("call", [_rope, _write, lambda *a: _rope(*a, in_place=True)])
def test_strides_of_outputs(call):
    for case in OVERLAPPING:
        assert call(*case) == W.ERR_SHAPE, case
    for case in APART:
        assert call(*case) == W.ERR_DEVICE, case
    assert call(4, 0, 512, 0) == (W.ERR_DEVICE if call is _write else W.OK)      # no heads to overlap


@pytest.mark.gpu
def test_expanded_outputs_are_refused():
    x = torch.randn((3, 4, 64), device="cuda").bfloat16()
    pos, table = torch.arange(3, device="cuda"), attn.rope_table(8, attn.rope_frequencies(64))
    cache = attn.kv_cache(1, 4, 64, 16)
    for out in (torch.empty((1, 4, 64), dtype=x.dtype, device="cuda").expand(3, 4, 64),
                torch.empty((3, 1, 64), dtype=x.dtype, device="cuda").expand(3, 4, 64)):
        for call in (lambda: attn.rope(x, pos, table, out=out), lambda: attn.rope(out, pos, table, out=out),
                     lambda: attn.kv_write(x, x, pos, cache, pos, table, q=x, q_out=out)):
            with pytest.raises(W.W4A16Error) as e:
                call()
            assert e.value.status == W.ERR_SHAPE
    # an input may be expanded, and an output lie in any order
    row = x[:1].expand(3, 4, 64)
    want = attn.rope(row.contiguous(), pos, table)
    assert torch.equal(attn.rope(row, pos, table), want)
    turned = torch.empty((4, 3, 64), dtype=x.dtype, device="cuda").transpose(0, 1)
    assert torch.equal(attn.rope(row, pos, table, out=turned), want)
