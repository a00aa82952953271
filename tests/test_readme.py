"""CPU test of the README's lines for a batch of requests: run as they stand, on plain lists in
place of the library, they leave every sequence with the tokens that it should have."""
import os
from types import SimpleNamespace

import numpy as np
import pytest

from oracle import batch_oracle as O

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


class Library:
    """paging, adapters and scoring on lists: a cache is a token's name for every slot."""

    def __init__(self, page, path, counts, news):
        self.page, self.path, self.counts, self.news = page, path, counts, news

    def page_pool(self, pages, rows, table_pages, page_size):
        self.pool = O.Pool([0] * pages, [[-1] * table_pages for _ in range(rows)], [0] * rows, self.page)
        self.pool.block_table = np.array(self.pool.table)
        return self.pool

    def cache_group(self, caches):
        self.caches = caches
        return caches

    def change(self, name, pool, a, b):
        out = getattr(pool, name)(list(a), list(b))
        pool.block_table = np.array(pool.table)
        assert all(out[0])
        return out

    def pages_resize(self, pool, rows, lens):
        return self.change("resize", pool, rows, lens)

    def pages_fork(self, pool, parents, children):
        return self.change("fork", pool, parents, children)

    def kv_copy_pages(self, group, src, dst):
        for s, d in zip(src, dst):
            if s >= 0:
                for cache in group:
                    cache[d] = list(cache[s])

    def slot(self, table, place):
        return table[place // self.page], place % self.page

    def write(self, row, places, names):
        for place, name in zip(places, names):
            page, at = self.slot(self.pool.table[row], place)
            assert self.pool.refs[page] == 1, "others see what is written"
            for cache in self.caches:
                cache[page][at] = name

    def text(self, row):
        at = [self.slot(self.pool.table[row], i) for i in range(self.pool.lens[row])]
        return [[cache[page][i] for page, i in at] for cache in self.caches]

    def verify_drafts(self, *args, **kw):
        # the layers' products have run: every new token is in the caches
        for b, n in enumerate(self.news):
            end = self.pool.lens[b]
            self.write(b, range(end - n, end), [f"new {b} {i}" for i in range(n)])
        return None, self.path, self.counts

    def kv_compact(self, group, table, lens, q_starts, path, counts):
        out = []
        for b, n in enumerate(lens):
            first = n - self.news[b]
            moves = O.compact(self.news[b], path[b], counts[b])
            for cache in group:
                for s, d in moves:
                    (p, i), (q, j) = self.slot(table[b], first + s), self.slot(table[b], first + d)
                    cache[q][j] = cache[p][i]
            out.append(first + len(moves))
        return np.array(out)


def block():
    text = open(README, encoding="utf-8").read()
    return next(x.split("```")[0] for x in text.split("```python\n")[1:] if "pages_fork" in x)


@pytest.mark.parametrize("prompts", [[16, 5, 30], [1, 15, 48]])
def test_the_lines_for_a_batch_leave_every_sequence_its_tokens(prompts):
    path, counts, news = [[0, 2, 5], [0, 7, -1], [0, 1, 2]], [3, 2, 1], [6, 8, 4]
    m = Library(16, path, counts, news)
    lines = block().splitlines(keepends=True)
    assert lines[0].startswith("from weight_only_int4_unpack_amd import")
    made = next(i for i, x in enumerate(lines) if "pages_resize" in x)
    none = SimpleNamespace(lora_plan=lambda *a, **k: None, lora=lambda *a, **k: None)
    lens = np.array(prompts) + news
    names = dict(paging=m, scoring=m, adapters=none, rows=np.arange(3), lens=lens, kv_lens=lens, parent_rows=[0, 2, 0],
                 child_rows=[3, 4, 5], caches=[[[None] * 16 for _ in range(1024)] for _ in range(2)])
    names.update({k: None for k in ("adapter_of_token x a b out scales logits ids q_starts max_q uniforms final_uniforms "
                                    "parents temperatures").split()})
    exec("".join(lines[1:made]), names)                  # the pool and the group
    m.pages_resize(m.pool, range(3), prompts)
    for b, n in enumerate(prompts):
        m.write(b, range(n), [f"prompt {b} {i}" for i in range(n)])
    exec("".join(lines[made:]), names)
    for row, b in enumerate([0, 1, 2, 0, 2, 0]):
        want = [f"prompt {b} {i}" for i in range(prompts[b])] + [f"new {b} {i}" for i in path[b][:counts[b]]]
        assert m.text(row) == [want] * 2
    for row in range(6):                                 # each goes on by itself
        end = m.pool.lens[row]
        m.kv_copy_pages(m.caches, *m.pages_resize(m.pool, [row], [end + 1])[1:])
        m.write(row, [end], [f"next {row}"])
    assert [t[0][-1] for t in map(m.text, range(6))] == [f"next {row}" for row in range(6)]
