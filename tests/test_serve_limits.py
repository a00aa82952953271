"""CPU tests of the largest calls: a grid of 256-thread workgroups holds fewer than 2^32
threads, so at most 2^24 - 1 workgroups. Beyond, a call is refused by its checks, not by
the launch."""
import pytest
import torch

from weight_only_int4_unpack_amd import attn, scoring
from weight_only_int4_unpack_amd import w4a16 as W

P = 0x10000                       # aligned, never dereferenced on the host
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")


def rope(heads, dim):             # two heads a lane group, 256 / (8, 16, 32) groups a workgroup
    return W.lib().w4a16_rope(attn._ROPE.pack(P, 2 * P, P, P, 1, 0, dim, 0, dim, 32, heads, dim, dim, 0, 0, 1), None)


def write(tokens, heads, dim):    # k's and v's, two a lane group
    return W.lib().w4a16_kv_write(attn._WRITE.pack(P, P, P, P, 4, 64, heads, dim, attn.KV_E4M3, P, P, P, 0, 0, 0, 0,
                                                   tokens, heads * dim, dim, heads * dim, dim, 0, 0, 0, 0, 0, 0, 0, 0,
                                                   1), None)


def read(tokens, heads, dim):     # four a lane group
    return W.lib().w4a16_kv_read(attn._READ.pack(P, P, P, P, 4, 64, heads, dim, attn.KV_E4M3, P, P, P, tokens, 1, 0),
                                 None)


def attend(sequences, heads):     # a workgroup for each sequence and head
    return W.lib().w4a16_tree_attention(attn._ATTEND.pack(
        P, P, 0, 0, 4, 64, heads, 128, attn.KV_SAME, P, P, P, P, P, P, 0, 4, heads * 128, 128, 1, sequences, 1, 1,
        heads, 0, 1, 0.1, 0), P, 1 << 40, None)


def score(tokens):                # a workgroup for each row
    return W.lib().w4a16_token_logprobs(scoring._ARGS.pack(P, P, P, P, 0, 0, tokens, 10, 10, 0, 1), P, 1 << 40, None)


MOST = (1 << 24) - 1


@pytest.mark.parametrize("call,most,step", [
    (lambda n: rope(n, 256), 2 * 8 * MOST, 2), (lambda n: rope(n, 128), 2 * 16 * MOST, 2),
    (lambda n: rope(n, 64), 2 * 32 * MOST, 2),
    (lambda n: write(n, 16, 256), MOST // 2, 1), (lambda n: read(n, 16, 256), MOST, 1),
    (lambda n: attend(n, 32), MOST // 32, 1), (score, MOST, 1),
])
def test_a_grid_holds_fewer_than_2_32_threads(call, most, step):
    assert call(most) == W.ERR_DEVICE
    assert call(most + step) == W.ERR_SHAPE
    assert call(2 * most) == W.ERR_SHAPE


def test_sizes_that_no_launch_takes_have_no_scratch_size():
    assert attn.tree_attention_workspace_bytes(MOST // 32, 1, 32, 32, 128) == 0
    for f in (lambda: attn.tree_attention_workspace_bytes(MOST // 32 + 1, 1, 32, 32, 128),
              lambda: scoring.workspace_bytes(MOST + 1, 1000, 0)):
        with pytest.raises(W.W4A16Error) as e:
            f()
        assert e.value.status == W.ERR_SHAPE
