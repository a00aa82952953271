"""GPU tests of forks and resizes of paged sequences, copies of pages, and compaction of an
accepted path, against plain Python lists. Everything here is whole numbers or copied bytes
and has to be equal."""
import numpy as np
import pytest
import torch

from oracle import batch_oracle as O
from weight_only_int4_unpack_amd import attn, batch_op, paging

pytestmark = pytest.mark.gpu
FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "fp16": torch.float16, "bf16": torch.bfloat16}


def ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def on_gpu(o, stride=None):
    wide = torch.full((len(o.table), stride or len(o.table[0])), 12345, dtype=torch.int32).cuda()
    table = wide[:, :len(o.table[0])]
    table.copy_(ints(o.table))
    return paging.PagePool(ints(o.refs), table, ints(o.lens), o.page), wide


def equal(pool, o):
    assert pool.refs.tolist() == o.refs
    assert pool.block_table.tolist() == o.table
    assert pool.lens.tolist() == o.lens


def lists(got):
    return tuple(x.tolist() for x in got)


def filled(g, pages, rows, entries, page):
    o = O.Pool([0] * pages, [[-1] * entries for _ in range(rows)], [0] * rows, page)
    order = list(g.permutation(pages))
    for r in range(rows):
        n = int(g.integers(0, entries * page // 2))
        k = -(-n // page)
        if k > len(order):
            break
        for j in range(k):
            o.table[r][j] = int(order.pop())
            o.refs[o.table[r][j]] = 1
        o.lens[r] = n
    return o


@pytest.mark.parametrize("page", [16, 64, 4096])
@pytest.mark.parametrize("seed", range(6))
def test_a_run_of_forks_and_resizes(seed, page):
    g = np.random.default_rng(seed)
    pages, rows, entries = [(40, 12, 7), (3000, 60, 40), (9, 5, 3)][seed % 3]
    o = filled(g, pages, rows, entries, page)
    pool, wide = on_gpu(o, entries + 3 * (seed % 2))
    refused = 0
    for step in range(12):
        n = int(g.integers(1, rows + 4))
        a, b = g.integers(-1, rows + 1, n).tolist(), g.integers(-1, rows + 1, n).tolist()
        if step % 3 == 0:
            got, want = paging.pages_fork(pool, ints(a), ints(b)), o.fork(a, b)
        else:
            room = entries * page
            lens = [int(x) for x in g.choice([0, 1, page, page + 1, room, room + 1, -1, int(g.integers(0, room))], n)]
            got, want = paging.pages_resize(pool, ints(a), ints(lens)), o.resize(a, lens)
        assert lists(got) == want
        equal(pool, o)
        refused += want[0].count(0)
    assert refused > 0
    assert (wide[:, entries:] == 12345).all()
    # the counts are what the tables say
    held = [p for row, n in zip(o.table, o.lens) for p in row[:-(-n // page)]]
    assert all(o.refs[p] == held.count(p) for p in range(pages))


def test_copy_on_write():
    o = O.Pool([0] * 8, [[-1] * 4 for _ in range(4)], [0] * 4, 16)
    pool, _ = on_gpu(o)
    steps = [("resize", [0], [40]),                       # 3 pages: 0, 1, 2
             ("fork", [0, 0], [1, 2]),                    # share 0 and 1, have 3 and 4 for 2
             ("resize", [1], [20]),                       # ends inside page 1, which others hold: 5 for it
             ("resize", [1, 2], [50, 24]),                # on from there: 3 and 6; 2 shrinks into page 1: 7 for it
             ("resize", [0], [64])]                       # a fourth: 4, which 2 gave back
    want = [([1], [-1], [-1]), ([1, 1], [2, 2], [3, 4]), ([1], [1], [5]), ([1, 1], [-1, 1], [-1, 7]), ([1], [-1], [-1])]
    for (kind, a, b), w in zip(steps, want):
        got = lists((paging.pages_fork if kind == "fork" else paging.pages_resize)(pool, ints(a), ints(b)))
        model = o.fork(a, b) if kind == "fork" else o.resize(a, b)
        assert got == model
        equal(pool, o)
        assert got == w
    assert o.table == [[0, 1, 2, 4], [0, 5, 3, 6], [0, 7, -1, -1], [-1] * 4]


def test_pages_given_out_lowest_first_in_the_order_of_the_list():
    o = O.Pool([0, 1, 0, 0, 1, 0, 0], [[-1] * 3 for _ in range(4)], [0] * 4, 16)
    pool, _ = on_gpu(o)
    # the third asks for more than is left, so that the fourth has to wait, while 0 needs none
    got = lists(paging.pages_resize(pool, ints([2, 0, 3, 1, 2]), ints([32, 16, 48, 16, 0])))
    assert got[0] == [1, 1, 0, 0, 0] and pool.block_table.tolist()[2] == [0, 2, -1]
    assert pool.block_table.tolist()[0] == [3, -1, -1] and pool.lens.tolist() == [16, 0, 32, 0]
    # what a call takes back is for the next
    got = lists(paging.pages_resize(pool, ints([2, 3]), ints([0, 48])))
    assert got[0] == [1, 0]
    got = lists(paging.pages_resize(pool, ints([3]), ints([48])))
    assert got[0] == [1] and pool.block_table.tolist()[3] == [0, 2, 5]


def test_a_long_list_and_a_large_pool():
    g = np.random.default_rng(5)
    o = O.Pool([0] * 100003, [[-1] * 20 for _ in range(4096)], [0] * 4096, 16)
    for p in g.choice(100003, 50000, replace=False):
        o.refs[p] = 1
    pool, _ = on_gpu(o)
    rows = g.permutation(4096).tolist()
    lens = g.integers(0, 321, 4096).tolist()
    assert lists(paging.pages_resize(pool, ints(rows), ints(lens))) == o.resize(rows, lens)
    equal(pool, o)
    half = g.permutation(4096)
    parents, children = half[:2048].tolist(), half[2048:].tolist()
    none = [0] * 2048
    assert lists(paging.pages_resize(pool, ints(children), ints(none))) == o.resize(children, none)
    assert lists(paging.pages_fork(pool, ints(parents), ints(children))) == o.fork(parents, children)
    equal(pool, o)


@pytest.mark.parametrize("others", [0, 1, 70])
def test_long_rows(others):
    # more pages than threads, one sequence or several at a time
    rows, entries, page = 4 + 2 * others, 5000, 16
    o = O.Pool([0] * 30000, [[-1] * entries for _ in range(rows)], [0] * rows, page)
    pool, _ = on_gpu(o)
    short = list(range(4, 4 + others))
    steps = [("resize", [0, 3, *short], [entries * page - 3, 2000 * page, *[37 * page + i for i in short]]),
             ("fork", [0, 3, *short], [1, 2, *[i + others for i in short]]),
             ("resize", [1, 0, *short], [1500 * page + 1, 0, *[5 * i for i in short]]),
             ("resize", [2, 3, 1], [0, 0, entries * page])]
    for kind, a, b in steps:
        got = (paging.pages_fork if kind == "fork" else paging.pages_resize)(pool, ints(a), ints(b))
        assert lists(got) == (o.fork(a, b) if kind == "fork" else o.resize(a, b))
        assert all(lists(got)[0])
        equal(pool, o)


def test_entries_that_are_no_pages():
    # a table with entries outside the pool: counted as no page, never followed
    o = O.Pool([1, 0, 0, 5], [[99, -7, 0], [3, 1 << 30, -1], [-1, -1, -1]], [40, 20, 0], 16)
    pool, _ = on_gpu(o)
    for kind, a, b in (("fork", [0], [2]), ("resize", [0, 1], [0, 17]), ("resize", [1, 2], [0, 0])):
        got = lists((paging.pages_fork if kind == "fork" else paging.pages_resize)(pool, ints(a), ints(b)))
        assert got == (o.fork(a, b) if kind == "fork" else o.resize(a, b))
        equal(pool, o)


def test_empty_lists_and_pools():
    pool = paging.page_pool(0, 2, 3, 16)
    assert lists(paging.pages_resize(pool, ints([0, 1]), ints([0, 5]))) == ([1, 0], [-1, -1], [-1, -1])
    assert lists(paging.pages_fork(pool, ints([0]), ints([1]))) == ([1], [-1], [-1])
    assert lists(paging.pages_fork(pool, ints([]), ints([]))) == ([], [], [])
    pool = paging.page_pool(4, 0, 3, 16)
    assert lists(paging.pages_resize(pool, ints([0]), ints([1]))) == ([0], [-1], [-1])
    with pytest.raises(RuntimeError, match="4096"):
        paging.pages_resize(paging.page_pool(4, 2, 3, 16), ints([0] * 4097), ints([0] * 4097))
    with pytest.raises(ValueError, match="lens"):
        paging.pages_resize(paging.page_pool(4, 2, 3, 16), ints([0]), ints([0, 1]))
    with pytest.raises(RuntimeError, match="power of two"):
        paging.pages_resize(paging.page_pool(4, 2, 3, 24), ints([0]), ints([0]))


# ---------------------------------------------------------------- copies and compaction
def caches(layers, pages, heads, dim, page, fmt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        c = attn.kv_cache(pages, heads, dim, page, FORMATS[fmt])
        for x in c:
            if x is not None:
                x.view(torch.uint8).random_(0, 120, generator=g)
        out.append(c)
    return out


def held(cs):
    return [[None if x is None else x.view(torch.uint8).clone() for x in c] for c in cs]


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("layers,pages,heads,dim,page", [(1, 5, 1, 16, 16), (3, 9, 5, 80, 16), (2, 6, 8, 128, 64),
                                                         (1, 4, 2, 256, 4096), (130, 5, 2, 64, 16)])
def test_copied_pages(fmt, layers, pages, heads, dim, page):
    cs = caches(layers, pages, heads, dim, page, fmt)
    want = held(cs)
    src, dst = [0, 3, -1, 2, 3, pages, 1], [1, 2, 0, -1, 3, 0, 1 << 30]
    for a, b in ((0, 1), (3, 2)):
        for layer in want:
            for x in layer:
                if x is not None:
                    x[b] = x[a]
    paging.kv_copy_pages(paging.cache_group(cs), ints(src), ints(dst))
    for c, w in zip(cs, want):
        for x, y in zip(c, w):
            assert y is None or torch.equal(x.view(torch.uint8), y)


def test_head_dims_of_8_and_odd_16_bit_rows():
    cs = caches(2, 4, 3, 8, 16, "bf16")
    want = held(cs)
    for layer in want:
        for x in layer[:2]:
            x[3] = x[1]
    paging.kv_copy_pages(paging.cache_group(cs), ints([1]), ints([3]))
    assert all(torch.equal(x.view(torch.uint8), y) for c, w in zip(cs, want) for x, y in zip(c[:2], w[:2]))


def compact_case(seed, batch, page, pages_each, heads, dim, fmt, layers, most=24):
    g = np.random.default_rng(seed)
    cs = caches(layers, batch * pages_each + 2, heads, dim, page, fmt, seed)
    news = [int(g.integers(1, most + 1)) for _ in range(batch)]
    lens = [int(g.integers(n, pages_each * page + 1)) for n in news]
    table = g.permutation(batch * pages_each + 2)[:batch * pages_each].reshape(batch, pages_each)
    width = max(news)
    path = np.full((batch, width), -1, np.int64)
    counts = []
    for b, n in enumerate(news):
        k = int(g.integers(1, n + 1))
        path[b, :k] = [0] + sorted(g.choice(np.arange(1, n), k - 1, replace=False).tolist()) if k > 1 else [0]
        counts.append(k)
    return cs, table, lens, news, path, counts


def moved(want, table, page, lens, news, path, counts):
    new = []
    pages = want[0][0].shape[0]
    for b, (n, length) in enumerate(zip(news, lens)):
        keep = O.compact(n, path[b].tolist(), counts[b]) if 0 < n <= length else None
        if keep is None:
            new.append(length)
            continue
        first = length - n
        new.append(first + len(keep))
        place = lambda t: (int(table[b][t // page]) if t // page < table.shape[1] else -1, t % page)   # noqa: E731
        for come, go in keep:
            (p, o), (q, r) = place(first + come), place(first + go)
            if 0 <= p < pages and 0 <= q < pages:
                for layer in want:
                    for x in layer:
                        if x is not None:
                            x[q, :, r] = x[p, :, o]
    return new


def by_head(cs):
    # [pages, heads, page, bytes] (a scale is 4 bytes)
    return [[None if x is None else x.view(torch.uint8).view(*x.shape[:3], -1).cpu().clone() for x in c] for c in cs]


def run_compact(cs, table, page, lens, news, path, counts, stride=None):
    starts = np.concatenate([[0], np.cumsum(news)])
    want = by_head(cs)
    new = moved(want, table, page, lens, news, path, counts)
    wide = torch.full((len(lens), stride or table.shape[1]), -1, dtype=torch.int32).cuda()
    wide[:, :table.shape[1]] = ints(table)
    got = paging.kv_compact(paging.cache_group(cs), wide[:, :table.shape[1]], ints(lens), ints(starts), ints(path),
                            ints(counts))
    assert got.tolist() == new
    for c, w in zip(by_head(cs), want):
        for x, y in zip(c, w):
            assert y is None or torch.equal(x, y)


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("batch,page,each,heads,dim,layers", [(1, 16, 4, 8, 128, 1), (5, 16, 9, 5, 80, 3),
                                                             (9, 64, 3, 2, 256, 2), (2, 16, 3, 40, 128, 2),
                                                             (3, 32, 2, 1, 64, 70)])
def test_compaction(fmt, batch, page, each, heads, dim, layers):
    for seed in range(3):
        cs, table, *rest = compact_case(seed, batch, page, each, heads, dim, fmt, layers)
        run_compact(cs, table, page, *rest, stride=each + seed)


def test_paths_longer_than_a_round():
    # more than 64 entries; tokens move by one place, every source being another's place
    cs = caches(2, 20, 2, 64, 16, "e4m3")
    table = np.random.default_rng(1).permutation(20).reshape(1, 20)
    for path in (list(range(1, 200)), [0] + list(range(2, 200)), list(range(0, 200, 2)), list(range(200))):
        run_compact(cs, table, 16, [300], [200], np.array([path + [-1] * (200 - len(path))]), [len(path)])


def test_paths_and_lengths_that_no_call_should_have():
    table = np.array([[0, 1, 2], [3, 99, 5], [6, -1, 8], [9, 10, 11], [12, 13, 14], [15, 16, 17], [18, 19, 20], [21, 22, 23]])
    lens = [40, 40, 40, 40, 5, -3, 70, 40]
    news = [10, 30, 30, 10, 9, 4, 50, 0]
    path = np.array([[0, 3, 3, 5, -1], [0, 4, 20, 25, 29], [1, 2, 18, 29, 30], [-1, 2, 3, 4, 5], [0, 2, 3, 4, 5],
                     [0, 1, 2, 3, 4], [3, 20, 30, 40, 49], [0, 1, 2, 3, 4]])
    counts = [5, 5, 99, 3, 2, 2, 5, 5]
    for fmt in ("bf16", "int8"):
        run_compact(caches(2, 24, 3, 64, 16, fmt), table, 16, lens, news, path, counts)
    for c in ([0] * 8, [-5] * 8, [1] * 8):
        run_compact(caches(1, 24, 3, 64, 16, "fp16"), table, 16, lens, news, path, c)


def test_compaction_without_caches_pages_or_sequences():
    none = paging.cache_group([attn.kv_cache(0, 2, 64, 16, torch.bfloat16)])
    got = paging.kv_compact(none, ints(np.zeros((2, 1))), ints([9, 7]), ints([0, 4, 6]), ints([[0, 2], [1, -1]]), ints([2, 1]))
    assert got.tolist() == [7, 6]
    assert paging.kv_compact(none, ints(np.zeros((0, 1))), ints([]), ints([0]), ints(np.zeros((0, 2))), ints([])).shape == (0,)
    paging.kv_copy_pages(none, ints([0]), ints([1]))
    paging.kv_copy_pages(none, ints([]), ints([]))


def test_offsets_past_32_bits():
    # a cache of more than 2^32 bytes: its last pages
    pages = 20000
    c = attn.KVCache(*(torch.empty((pages, 8, 64, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    assert c.k.numel() * 2 > 1 << 32
    for x in c[:2]:
        x[pages - 3:] = torch.randn((3, 8, 64, 256), device="cuda").bfloat16()
    want = [x[pages - 2].clone() for x in c[:2]]
    group = paging.cache_group([c])
    paging.kv_copy_pages(group, ints([pages - 2]), ints([pages - 1]))
    assert all(torch.equal(x[pages - 1], w) for x, w in zip(c[:2], want))
    paging.kv_compact(group, ints([[pages - 2]]), ints([64]), ints([0, 10]), ints([[0, 9]]), ints([2]))
    assert all(torch.equal(x[pages - 2, :, 55], w[:, 63]) for x, w in zip(c[:2], want))


def test_refused_groups():
    a, b = attn.kv_cache(4, 2, 64, 16), attn.kv_cache(4, 2, 64, 32)
    with pytest.raises(ValueError, match="one shape and dtype"):
        paging.cache_group([a, b])
    with pytest.raises(ValueError, match="one shape and dtype"):
        paging.cache_group([attn.kv_cache(4, 2, 64, 16, torch.float16), attn.kv_cache(4, 2, 64, 16, torch.bfloat16)])
    group = paging.cache_group([a])
    with pytest.raises(ValueError, match="dst"):
        paging.kv_copy_pages(group, ints([1]), ints([1, 2]))
    with pytest.raises(RuntimeError, match="block_table"):
        paging.kv_compact(group, ints([[0, 1]]).expand(2, 2), ints([1, 1]), ints([0, 1, 2]), ints([[0], [0]]), ints([1, 1]))


def test_captured_and_replayed():
    # a beam step: continuations dropped, forked anew, their pages copied; and a compaction
    o = O.Pool([0] * 64, [[-1] * 4 for _ in range(6)], [0] * 6, 16)
    pool, _ = on_gpu(o)
    paging.pages_resize(pool, ints([0, 1, 2]), ints([40, 9, 33]))
    o.resize([0, 1, 2], [40, 9, 33])
    cs = caches(3, 64, 2, 64, 16, "e4m3")
    group = paging.cache_group(cs)
    parents, children, zero = ints([0, 1, 2]), ints([3, 4, 5]), ints([0, 0, 0])
    starts, path, counts = ints([0, 8, 10, 20]), ints([[0, 3, 7], [0, 1, -1], [0, 5, 9]]), ints([3, 2, 3])

    def step():
        paging.pages_resize(pool, children, zero)
        served, src, dst = paging.pages_fork(pool, parents, children)
        paging.kv_copy_pages(group, src, dst)
        return served, src, dst, paging.kv_compact(group, pool.block_table[3:], pool.lens[3:], starts, path, counts)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
    for turn, order in enumerate(([0, 1, 2], [2, 0, 1], [1, 1, 1], [0, 1, 2])):
        parents.copy_(ints(order))
        torch.cuda.synchronize()
        want = by_head(cs)
        o.resize([3, 4, 5], [0, 0, 0])
        served, src, dst = o.fork(order, [3, 4, 5])
        for a, b in zip(src, dst):
            if a >= 0:
                for layer in want:
                    for x in layer:
                        if x is not None:
                            x[b] = x[a]
        new = moved(want, np.array(o.table[3:]), 16, o.lens[3:], [8, 2, 10], path.cpu().numpy(), counts.tolist())
        graph.replay()
        torch.cuda.synchronize()
        assert lists(out[:3]) == (served, src, dst) and out[3].tolist() == new
        equal(pool, o)
        for c, w in zip(by_head(cs), want):
            for x, y in zip(c, w):
                assert y is None or torch.equal(x, y)
        torch.zeros(1000, device="cuda").sum().item()    # eager work between the replays


def test_lists_that_are_views_of_the_pool():
    # the parents of rows 1 and 2 stand in their own lengths, which the call changes: 0, then 40
    o = O.Pool([0] * 12, [[-1] * 4 for _ in range(5)], [0] * 5, 16)
    pool, _ = on_gpu(o)
    paging.pages_resize(pool, ints([0, 3]), ints([40, 5]))
    o.resize([0, 3], [40, 5])
    got = lists(paging.pages_fork(pool, pool.lens[1:3], ints([1, 2])))
    assert got == o.fork([0, 0], [1, 2]) and got[0] == [1, 1]
    equal(pool, o)
    # every row at the length that it has: those that share a partly filled page get their own
    assert lists(paging.pages_resize(pool, ints(range(5)), pool.lens)) == o.resize(list(range(5)), list(o.lens))
    equal(pool, o)
    # row 4 is empty: its length is the number of the row to be freed
    assert lists(paging.pages_resize(pool, pool.lens[4:], ints([0]))) == o.resize([0], [0])
    equal(pool, o)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_arrays_that_share_memory_are_copied_but_not_compacted(fmt):
    # one workgroup would move what another has moved already
    c, d = caches(2, 6, 2, 64, 16, fmt)
    part = lambda x, i: None if x is None else x[i:i + 3]                            # noqa: E731
    cut = lambda i: attn.KVCache(*(part(x, i) for x in c))                           # noqa: E731
    args = ints([[0, 1, 2]]), ints([40]), ints([0, 30]), ints([list(range(1, 13))]), ints([12])
    for shared in ([c, c], [c, d, c], [c, d._replace(v=c.k)], [c._replace(v=c.k)], [cut(0), cut(2)]):
        group = paging.cache_group(shared)
        assert not group.apart
        with pytest.raises(ValueError, match="share memory"):
            paging.kv_compact(group, *args)
        with pytest.raises(ValueError, match="share memory"):
            batch_op.kv_compact(group, *args)
    if fmt == "e4m3":
        assert not paging.cache_group([c, d._replace(k_scale=c.v_scale)]).apart
    paging.kv_copy_pages(paging.cache_group([c, c]), ints([1]), ints([4]))
    assert all(torch.equal(x[1].view(torch.uint8), x[4].view(torch.uint8)) for x in c if x is not None)
    # halves of one array lie side by side
    assert paging.cache_group([cut(0), cut(3)]).apart
    run_compact([cut(0), cut(3)], np.array([[2, 0, 1]]), 16, [40], [30], np.array([list(range(1, 13))]), [12])
