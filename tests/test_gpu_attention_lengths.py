"""GPU tests of attention where a sequence has more new tokens than max_q, or more
cached ones than its table has pages for."""
import pytest
import torch

from attention_case import Strict
from test_gpu_tree_attention import ancestors, random_trees
from weight_only_int4_unpack_amd import attn

pytestmark = pytest.mark.gpu
FORMATS = [("16", torch.bfloat16), ("e4m3", torch.bfloat16), ("int8", torch.float16)]


def say(*a):
    print(*a, flush=True)


class Cut(Strict):
    """Computes the first max_q new tokens of each sequence only."""
    max_q = None

    def run(self, mask=None, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        got = attn.tree_attention(self.q, self.cache, self.table, self.kv_lens, self.starts, self.max_q,
                                  mask=mask, scale=self.scale, out=out, lse=lse)
        at = 0
        for n in self.news:                     # the others stay as they are: taken out here
            assert bool((out[at + self.max_q:at + n] == 7.0).all()) and bool((lse[at + self.max_q:at + n] == 7.0).all())
            at += n
        return got

    def check_first(self, out, lse, rows=None):
        """The rows that are computed, against all rows' oracle."""
        at = 0
        whole, wl = attn.tree_attention(self.q, self.cache, self.table, self.kv_lens, self.starts, max(self.news),
                                        mask=rows and rows[1], scale=self.scale)
        for n in self.news:
            out[at + self.max_q:at + n] = whole[at + self.max_q:at + n]
            lse[at + self.max_q:at + n] = wl[at + self.max_q:at + n]
            at += n
        self.check(out, lse, rows=rows and rows[0])


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("max_q,news", [(1, [3, 1, 40]), (2, [3, 9, 2]), (9, [20, 10, 9]), (20, [21, 90, 20]),
                                        (33, [70, 33, 34])])
def test_more_new_tokens_than_max_q(max_q, news, fmt, dtype):
    # new token i still sees what comes before the new ones and the new ones up to itself
    say("max_q", max_q, news, fmt, dtype)
    c = Cut([200, 131, 64 + 26], news, 4, 2, 64, fmt, dtype, 16, seed=41)
    c.max_q = max_q
    c.check_first(*c.run())
    trees = random_trees(news, 5)
    mask = attn.tree_mask(trees)
    c.check_first(*c.run(mask=mask), rows=([ancestors(t) for t in trees], mask))


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("news", [[1, 1], [5, 3], [20, 12], [40, 70]])
def test_more_cached_tokens_than_the_table_holds(news, fmt, dtype):
    # what lies past the table's last page is seen by none; the new ones stay where they are,
    # the last of all: with 48 of 100 tokens on pages, every new token sees all 48
    say("short table", news, fmt, dtype)
    c = Strict([100, 90], news, 4, 2, 64, fmt, dtype, 16, seed=42)
    c.table = c.table[:, :3].contiguous()
    c.check(*c.run(), held=48)
    trees = random_trees(news, 6)
    c.check(*c.run(mask=attn.tree_mask(trees)), rows=[ancestors(t) for t in trees], held=48)
