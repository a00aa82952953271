"""GPU tests of the verification of drafted tokens against the fp64 oracle. Results are whole
numbers and have to be equal: both sides sum in fp64, whose order moves a border by some
2^-50 of the sum, and a random number of 24 bits meets one of 2^17 borders to that with
a probability below 2^-30."""
import math

import numpy as np
import pytest
import torch

from oracle import batch_oracle as O
from weight_only_int4_unpack_amd import scoring

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def cuda(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


def make(seed, news, vocab, dtype="bf16", tree=False, probs=False, temps=None, pad=0, spread=2.0):
    """Random sequences whose drafts are often right; rows `pad` logits apart."""
    g = np.random.default_rng(seed)
    T = sum(news)
    x = (g.standard_normal((T, vocab)) * spread).astype(np.float32)
    liked = g.integers(0, vocab, (T, 3))
    x[np.arange(T)[:, None], liked] += math.log(vocab) + spread ** 2 / 2 + np.array([2.0, 1.0, 0.0])
    wide = torch.zeros((T, vocab + pad), dtype=DT[dtype])
    wide[:, :vocab] = torch.from_numpy(x).to(DT[dtype])
    logits = wide.cuda()[:, :vocab]
    held = logits.float().cpu().numpy()
    starts = np.concatenate([[0], np.cumsum(news)])
    parents, ids = [], []
    for b, n in enumerate(news):
        for i in range(n):
            p = -1 if i == 0 else int(g.integers(0, i)) if tree else i - 1
            parents.append(p)
            ids.append(int(liked[starts[b] + p, g.integers(0, 3)]) if p >= 0 else int(g.integers(0, vocab)))
    q = None
    if probs:
        q = held.astype(np.float64) + g.standard_normal((T, vocab))
        q = np.exp(q - q.max(-1, keepdims=True))
        q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    u, final = g.random(T).astype(np.float32), g.random(len(news)).astype(np.float32)
    u, final = np.minimum(u, np.float32(1 - 2.0 ** -24)), np.minimum(final, np.float32(1 - 2.0 ** -24))
    return dict(logits=logits, held=held, starts=starts, parents=parents, ids=ids, q=q, u=u, final=final, tree=tree,
                temps=temps, news=news)


def call(c, max_q=None, **kw):
    a = dict(parents=cuda(c["parents"], torch.int32) if c["tree"] else None,
             draft_probs=None if c["q"] is None else cuda(c["q"]),
             temperatures=None if c["temps"] is None else cuda(c["temps"], torch.float32))
    a.update(kw)
    return scoring.verify_drafts(c["logits"], cuda(c["ids"], torch.int64), cuda(c["starts"], torch.int32),
                                 max(c["news"]) if max_q is None else max_q, cuda(c["u"]), cuda(c["final"]), **a)


def want(c, max_q=None):
    max_q = max(c["news"]) if max_q is None else max_q
    out = []
    for b in range(len(c["news"])):
        lo, n = c["starts"][b], min(c["news"][b], max_q)
        if n == 0:
            out.append(([], []))
            continue
        at = slice(lo, lo + n)
        out.append(O.verify(c["held"][at], c["ids"][at], c["parents"][at], c["u"][at], c["final"][b],
                            None if c["q"] is None else c["q"][at], 1.0 if c["temps"] is None else float(np.float32(c["temps"][b]))))
    fill = lambda v: v + [-1] * (max_q - len(v))                                    # noqa: E731
    return [fill(t) for t, _ in out], [fill(p) for _, p in out], [len(p) for _, p in out]


def same(got, expected):
    assert got[2].tolist() == expected[2]
    assert got[1].tolist() == expected[1]
    assert got[0].tolist() == expected[0]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 1017, 1024, 1025, 2041, 2048, 2049, 5003, 32000])
def test_against_the_oracle(vocab, mode, dtype):
    c = make(vocab * 3 + len(mode), [3, 1, 0, 7, 2, 5], vocab, dtype, mode == "tree", mode == "drawn",
             temps=[1.0, 0.7, 1.0, 0.0, 1.3, 0.25])
    same(call(c), want(c))


@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
@pytest.mark.parametrize("pad", [0, 1, 5, 13])
def test_rows_that_lie_apart_and_large_vocabularies(mode, pad):
    for seed in range(4):
        c = make(seed, [4, 6, 1, 3], 151667, "bf16", mode == "tree", mode == "drawn", pad=pad)
        same(call(c), want(c))


def test_rows_of_draft_probabilities_that_lie_apart():
    c = make(5, [4, 6, 1, 3], 3001, "fp16", probs=True)
    wide = torch.zeros((14, 3010)).cuda()
    wide[:, 3:3004] = cuda(c["q"])
    same(call(c, draft_probs=wide[:, 3:3004]), want(c))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
def test_rows_of_more_spans_than_a_sequence_has_waves(mode, dtype):
    # 96 to 600 sequences leave each 5 workgroups to one, of 8 waves, for 20 spans of 1024
    for seed, sequences in enumerate((96, 250, 600)):
        g = np.random.default_rng(seed)
        news = [int(n) for n in g.integers(1, 4, sequences)]
        c = make(seed + 30, news, 20003, dtype, mode == "tree", mode == "drawn", temps=list(g.choice([0.7, 1.0], sequences)))
        same(call(c), want(c))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("mode", ["given", "drawn"])
def test_the_largest_vocabulary_and_most_nodes(mode, dtype):
    c = make(8, [3, 0, 5], 1 << 20, dtype, False, mode == "drawn", temps=[1.0, 1.0, 0.5], pad=3)
    same(call(c, max_q=1024), want(c, max_q=1024))


@pytest.mark.parametrize("mode", ["given", "drawn"])
def test_offsets_past_32_bits(mode):
    # the last sequence's rows lie past 2^31 logits (and probabilities): as the same rows alone
    c = make(7, [4, 4], 151667, "bf16", False, mode == "drawn")
    T, V = 14400, 151667
    logits = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    assert (T - 4) * V > 1 << 31
    place = lambda x: torch.cat([x[:4], x.new_zeros((T - 8, *x.shape[1:])), x[4:]])                   # noqa: E731
    logits[:4], logits[-4:] = c["logits"][:4], c["logits"][4:]
    probs = None if c["q"] is None else place(cuda(c["q"]))
    got = scoring.verify_drafts(logits, place(cuda(c["ids"], torch.int64)), cuda([0, 4, T - 4, T], torch.int32), 4,
                                place(cuda(c["u"])), cuda([c["final"][0], 0.5, c["final"][1]]), draft_probs=probs)
    same([x[[0, 2]] for x in got], want(c))


@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
def test_many_sequences(mode):
    # more than the second kernel's workgroups of a sequence share, and more than one look at q_starts
    g = np.random.default_rng(1)
    news = [int(n) for n in g.integers(0, 6, 5000)]
    c = make(2, news, 67, "fp32", mode == "tree", mode == "drawn", temps=list(g.choice([0.0, 0.5, 1.0], 5000)))
    same(call(c), want(c))


def test_long_trees_and_chains():
    for tree in (False, True):
        # weights of one token only: chains are accepted to their ends
        c = make(3, [1024, 700, 65, 64], 300, "fp16", tree, spread=1.0)
        same(call(c), want(c))
    c = make(4, [300], 40, "fp32")
    c["ids"] = [int(np.argmax(c["held"][max(i - 1, 0)])) for i in range(300)]
    c["temps"] = [0.0]
    got = call(c)
    same(got, want(c))
    assert got[2].tolist() == [300]


def test_nodes_past_max_q_are_as_if_not_drafted():
    c = make(6, [9, 4, 2], 500, "bf16", tree=True)
    for max_q in (1, 3, 9, 20):
        same(call(c, max_q), want(c, max_q))
    got = call(c, 0)
    assert got[0].shape == (3, 0) and got[2].tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", sorted(DT))
def test_masked_logits(dtype):
    low = float(torch.finfo(DT[dtype]).min)
    for mode in ("given", "drawn"):
        c = make(7, [3, 3, 3, 3], 2100, dtype, probs=mode == "drawn")
        keep = torch.zeros(2100, dtype=torch.bool).cuda()
        keep[[5, 17, 2050]] = True
        c["logits"][:3, ~keep] = -math.inf           # three left
        c["logits"][3:6, ~keep] = low                # the same by the lowest value
        c["logits"][6:9] = -math.inf
        c["logits"][6:9, 2099] = -3.0                # one left
        c["logits"][9:12] = low                      # all alike
        c["held"] = c["logits"].float().cpu().numpy()
        for i in range(12):
            c["ids"][i] = [5, 17, 2099, 4][(i * 7) % 4]
        same(call(c), want(c))


@pytest.mark.parametrize("bad", [math.nan, math.inf, "all -inf"])
@pytest.mark.parametrize("greedy", [False, True])
def test_a_row_without_a_softmax_ends_its_sequence(bad, greedy):
    c = make(8, [3, 3], 900, "fp32", temps=[0.0 if greedy else 1.0] * 2)
    for b in range(2):
        c["ids"][3 * b + 1] = int(np.argmax(c["held"][3 * b]))
    c["u"][:] = 0.0                                  # every draft that can be is accepted
    if bad == "all -inf":
        c["logits"][1] = -math.inf
    else:
        c["logits"][1, 899] = bad
    c["held"] = c["logits"].float().cpu().numpy()
    got = call(c)
    same(got, want(c))
    assert got[0][0].tolist() == [c["ids"][1], -1, -1] and got[2][0] == 2


def test_greedy_ties_go_to_the_lowest_index():
    x = torch.full((2, 5000), -1.0, dtype=torch.bfloat16)
    x[:, [77, 78, 2049, 4999]] = 3.0
    ids, starts, u, f = cuda([0, 77]), cuda([0, 2], torch.int32), cuda([0.5, 0.99]), cuda([0.999])
    for q in (None, torch.full((2, 5000), 1 / 5000).cuda()):
        t, p, n = scoring.verify_drafts(x.cuda(), ids, starts, 2, u, f, draft_probs=q, temperatures=cuda([0.0]))
        assert t.tolist() == [[77, 77]] and n.tolist() == [2]
        t, p, n = scoring.verify_drafts(x.cuda(), cuda([0, 78]), starts, 2, u, f, draft_probs=q, temperatures=cuda([0.0]))
        assert t.tolist() == [[77, -1]] and p.tolist() == [[0, -1]]


@pytest.mark.parametrize("t", [-1.0, math.nan, -0.0])
def test_what_is_not_above_zero_is_greedy(t):
    c = make(9, [4], 1000, temps=[t])
    a = call(c)
    c["temps"] = [0.0]
    same(a, want(c))


def test_extreme_temperatures():
    c = make(10, [4, 4, 4], 3000, "fp32", temps=[1e-45, 1e30, math.inf])
    c["logits"][:, 1000:] = -math.inf
    c["held"] = c["logits"].cpu().numpy()
    same(call(c), want(c))


def test_borders_by_arithmetic():
    # four equal weights: p = 1/4 each, and every number here is exact
    x = torch.zeros((2, 4)).cuda()
    starts = cuda([0, 2], torch.int32)

    def run(u, f, q=None, token=2):
        probs = None if q is None else cuda([q, q], torch.float32)
        t, _, n = scoring.verify_drafts(x, cuda([0, token]), starts, 2, cuda([0.0, u]), cuda([f]), draft_probs=probs)
        return t[0, :int(n)].tolist()
    below = 0.25 - 2.0 ** -26
    assert run(below, 0.0) == [2, 0] and run(0.25, 0.0) == [0]          # u < p, not u <= p
    # rejected: three left, a third each; borders at 1/3 and 2/3
    assert [run(0.9, f) for f in (0.33, 0.34, 0.66, 0.67, 0.999)] == [[0], [1], [1], [3], [3]]
    # drawn from q: accepted if u q < p
    q = [0.25, 0.0, 0.5, 0.25]
    assert run(0.5 - 2.0 ** -25, 0.0, q) == [2, 0] and run(0.5, 0.0, q) == [1]
    # above the draft: (0, 1/4, 0, 0)
    assert [run(0.9, f, q) for f in (0.0, 0.5, 0.999)] == [[1]] * 3
    # after an accepted token: a draw from p, borders at multiples of 1/4 that belong to the right
    assert [run(0.0, f)[1] for f in (0.0, below, 0.25, 0.5, 0.75, 1 - 2.0 ** -24)] == [0, 0, 1, 2, 3, 3]
    # the draft is the model: always accepted; were it not, nothing is left, and the draw is the model's
    same_q = [0.25] * 4
    assert run(1 - 2.0 ** -24, 0.6, same_q) == [2, 2] and run(1.0, 0.6, same_q) == [2]


def test_siblings_and_tokens_that_cannot_be():
    x = torch.zeros((5, 4)).cuda()
    starts = cuda([0, 5], torch.int32)

    def run(ids, u, f, parents=(-1, 0, 0, 0, 0)):
        t, p, n = scoring.verify_drafts(x, cuda(ids), starts, 5, cuda(u), cuda([f]), parents=cuda(list(parents), torch.int32))
        n = int(n)
        return t[0, :n].tolist(), p[0, :n].tolist()
    # rejected at 1/4, then at 1/3, then accepted at 1/2 (weights 1 of 2 left)
    assert run([0, 3, 1, 0, 2], [0, 0.3, 0.4, 0.45, 0.0], 0.0) == ([0, 0], [0, 3])
    # the same token twice: the second is rejected whatever its number, and costs nothing
    assert run([0, 3, 3, 1, 2], [0, 0.3, 0.0, 0.3, 0.0], 0.0) == ([1, 0], [0, 3])
    # all four tokens rejected (by numbers that are not below 1): the remainder is empty
    assert run([0, 3, 1, 0, 2], [0, 1.0, 1.0, 1.0, 1.0], 0.5) == ([2], [0])
    # tokens outside the vocabulary are never accepted
    assert run([0, -1, 4, 1 << 40, -(1 << 40)], [0.0] * 5, 0.0) == ([0], [0])
    # parents that are not before a node: never reached
    assert run([0, 1, 1, 1, 1], [0.0] * 5, 0.0, (0, 1, 3, -1, 99)) == ([0], [0])
    # NaN for a random number: not accepted; the draw takes the last token that there is
    assert run([0, 1, 2, 3, 0], [math.nan] * 5, math.nan, (-1, 0, 1, 2, 3)) == ([3], [0])


def test_not_a_number_in_the_draft_counts_as_nothing_above_it():
    c = make(11, [3, 2], 600, "fp32", probs=True)
    c["u"][:] = 1.0
    c["q"][:, 100:] = math.nan
    same(call(c), want(c))


def test_lengths_that_no_call_should_have():
    # q_starts outside the rows, and falling: nothing is read outside, other sequences are as they are
    c = make(12, [3, 3, 2], 400)
    good = want(c)
    for starts in ([0, 3, 6, 99], [-5, 3, 6, 8], [0, 3, 1, 8]):
        c["starts"] = starts
        t, p, n = call(c, 3)
        assert t[0].tolist() == good[0][0] and p[0].tolist() == good[1][0]
        assert 0 <= int(n.min()) and int(n.max()) <= 3
    none = scoring.verify_drafts(c["logits"][:0], cuda([], torch.int64), cuda([0, 0, 0], torch.int32), 2,
                                 cuda([], torch.float32), cuda([0.5, 0.5]))
    assert none[0].tolist() == [[-1, -1]] * 2 and none[2].tolist() == [0, 0]
    empty = scoring.verify_drafts(c["logits"], cuda(c["ids"]), cuda([0], torch.int32), 2, cuda(c["u"]),
                                  cuda([], torch.float32))
    assert empty[0].shape == (0, 2) and empty[2].shape == (0,)


@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
def test_tokens_are_distributed_as_the_models(mode):
    # The first token that comes out of N independent sequences is a draw from p: its counts are
    # binomial, and 5 standard deviations of one of 10 tokens are missed with probability 6e-6.
    g = np.random.default_rng(13)
    N, V = 40000, 10
    x = torch.from_numpy(g.standard_normal(V).astype(np.float32)).cuda()
    p = torch.softmax(x.double() / 0.8, 0).cpu().numpy()
    n = 4 if mode == "tree" else 2
    q = torch.softmax(torch.from_numpy(g.standard_normal(V).astype(np.float32)), 0)
    ids = np.zeros((N, n), np.int64)
    if mode == "tree":
        ids[:, 1:] = [3, 7, 1]
    else:
        ids[:, 1] = torch.multinomial(q, N, True, generator=torch.Generator().manual_seed(1)).numpy() if mode == "drawn" else 3
    t, _, _ = scoring.verify_drafts(
        x.expand(N * n, V), cuda(ids.reshape(-1)), cuda(np.arange(N + 1) * n, torch.int32), n,
        cuda(g.random(N * n, dtype=np.float32)), cuda(g.random(N, dtype=np.float32)),
        parents=cuda(np.tile([-1, 0, 0, 0], N), torch.int32) if mode == "tree" else None,
        draft_probs=q.cuda().expand(N * n, V) if mode == "drawn" else None, temperatures=torch.full((N,), 0.8).cuda())
    counts = np.bincount(t[:, 0].cpu().numpy(), minlength=V)
    assert (np.abs(counts - N * p) < 5 * np.sqrt(N * p * (1 - p)) + 1).all()


@pytest.mark.parametrize("mode", ["tree", "drawn"])
def test_captured_and_replayed_with_new_inputs(mode):
    kw = dict(tree=mode == "tree", probs=mode == "drawn", temps=[1.0, 0.0, 0.6, 1.0])
    cases = [make(s, [4, 2, 6, 3], 20011, "bf16", **kw) for s in (20, 21, 22)]
    held = dict(logits=cases[0]["logits"].clone(), ids=cuda(cases[0]["ids"]), u=cuda(cases[0]["u"]),
                final=cuda(cases[0]["final"]), starts=cuda(cases[0]["starts"], torch.int32),
                parents=cuda(cases[0]["parents"], torch.int32), q=None if mode == "tree" else cuda(cases[0]["q"]))

    def step():
        return scoring.verify_drafts(held["logits"], held["ids"], held["starts"], 6, held["u"], held["final"],
                                     parents=held["parents"] if mode == "tree" else None, draft_probs=held["q"],
                                     temperatures=cuda_temps)
    cuda_temps = cuda(cases[0]["temps"], torch.float32)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
    for turn in range(2):
        for c in cases:
            held["logits"].copy_(c["logits"])
            for name in ("ids", "u", "final"):
                held[name].copy_(cuda(c[name]))
            held["parents"].copy_(cuda(c["parents"], torch.int32))
            if mode == "drawn":
                held["q"].copy_(cuda(c["q"]))
            graph.replay()
            torch.cuda.synchronize()
            same(out, want(c))
            same(call(c), want(c))                   # eager work between the replays


def test_two_streams_at_once():
    cases = [make(s, [6] * 40, 30011, "bf16", probs=True) for s in (30, 31)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for turn in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append((c, call(c)))
    torch.cuda.synchronize()
    for c, o in outs:
        same(o, want(c))


def test_refusals():
    c = make(1, [2, 2], 64)
    for kw, what in ((dict(parents=cuda([0, 0, 0, 0], torch.int32), draft_probs=torch.zeros((4, 64)).cuda()), "chains"),
                     (dict(draft_probs=torch.zeros((4, 63)).cuda()), "draft_probs"),
                     (dict(draft_probs=torch.zeros((4, 64)).cuda().half()), "draft_probs"),
                     (dict(temperatures=torch.zeros(3).cuda()), "temperatures"),
                     (dict(parents=cuda([0, 0, 0, 0], torch.int64)), "parents")):
        with pytest.raises(ValueError, match=what):
            call(c, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        scoring.verify_drafts(c["logits"].t().contiguous().t(), cuda(c["ids"]), cuda(c["starts"], torch.int32), 2,
                              cuda(c["u"]), cuda(c["final"]))
    with pytest.raises(RuntimeError, match="1024"):
        call(c, 1025)
    with pytest.raises(RuntimeError, match="2\\^20"):
        scoring.verify_drafts(torch.zeros((1, (1 << 20) + 1), dtype=torch.bfloat16).cuda(), cuda([0]),
                              cuda([0, 1], torch.int32), 1, cuda([0.0]), cuda([0.0]))


# Rows that are summed again: where a random number is next to the border that it is compared with (fp32 sums
# cannot tell), and where the draft follows the model so closely that little but roundings remains.
def beside_borders(c, seed, accept):
    """Sets each random number on the walk to the fp32 number below the oracle's border (the token is accepted) or to
    the one from the border on (it is not), as accept() says; a walk ends where it says no to all of a node's."""
    g, last = np.random.default_rng(seed), np.float32(1 - 2.0 ** -24)
    for b, n in enumerate(c["news"]):
        lo, node = c["starts"][b], 0
        while node is not None:
            w = O.weights(c["held"][lo + node], 1.0 if c["temps"] is None else float(np.float32(c["temps"][b])))
            left, gone, at, node = w.sum(), [], node, None
            for k in range(at + 1, n):
                if c["parents"][lo + k] != at or c["ids"][lo + k] in gone:
                    continue
                t = c["ids"][lo + k]
                q = 1.0 if c["q"] is None else float(c["q"][lo + at, t])
                border = float(w[t] / (left * q))
                up = np.float32(border)
                up = up if float(up) >= border else np.nextafter(up, np.float32(2), dtype=np.float32)
                if border > float(last) or accept(g):
                    c["u"][lo + k] = min(np.nextafter(up, np.float32(0), dtype=np.float32), last)
                    node = k
                    break
                c["u"][lo + k] = up
                if c["q"] is not None:
                    break
                gone.append(t)
                left -= w[t]
    return c


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("mode", ["given", "tree", "drawn"])
@pytest.mark.parametrize("vocab,sequences,pad", [(20003, 1, 0), (20003, 40, 3), (20003, 300, 0), (151667, 1, 5), (151667, 6, 0),
                                                 (1 << 20, 1, 0)])
def test_random_numbers_beside_the_borders_of_large_rows(vocab, sequences, pad, mode, dtype):
    news = [6] if sequences == 1 else [2 + b % 5 if sequences < 300 else 2 + b % 2 for b in range(sequences)]
    temps = None if sequences == 6 else [0.8, 1.0, 1.7][:len(news)] + [1.0] * (len(news) - 3)
    for seed, share in ((0, 1.0), (1, 0.7), (2, 0.0))[:1 if vocab == 1 << 20 else 3]:
        c = make(seed, news, vocab, dtype, mode == "tree", mode == "drawn", temps, pad)
        beside_borders(c, seed, lambda g: g.random() < share)
        got = call(c)
        same(got, want(c))
        if mode == "given" and share in (0.0, 1.0):
            assert got[2].tolist() == (news if share else [1] * sequences)


def follows(seed, vocab, dtype, draws, temperature):
    """`draws` sequences of one drafted token, which is rejected: the draft is the model's distribution as fp32 numbers but
    for two tokens, one with more and, at the end, one with less. Below the latter lies what fp32 rounded away, token
    by token, and final random numbers in the middle of a token's share of it."""
    c = make(seed, [2], vocab, dtype, temps=[temperature])
    held = c["held"][0]
    for t in (vocab // 3, vocab - 2):
        held[t] = held.max() if t == vocab // 3 else held[vocab // 3]
    c["logits"][0] = torch.from_numpy(held)
    c["held"][0] = c["logits"][0].float().cpu().numpy()
    p = O.weights(c["held"][0], float(np.float32(temperature)))
    p /= p.sum()
    q = p.astype(np.float32)
    q[vocab // 3] += np.float32(0.25)
    q[vocab - 2] = 0.0
    r = np.fmax(p - q.astype(np.float64), 0.0)
    up = np.cumsum(r)
    # shares that final numbers of 24 bits can name, and that are wider than what both sides' sums differ by
    places = np.flatnonzero(r / 2 > up * 2.0 ** -24 + np.cumsum(p) * 2.0 ** -45)
    first, wide = int(np.flatnonzero(r)[0]), vocab - 2
    assert r[first] > p[first] * 2.0 ** -44
    picks = [first, wide, *np.random.default_rng(seed).choice(places, draws - 2)]
    final = np.array([(up[t] - r[t] / 2) / up[-1] for t in picks]).astype(np.float32)
    final[0] = 0.0
    c.update(news=[2] * draws, starts=np.arange(draws + 1) * 2, parents=[-1, 0] * draws, ids=[0, vocab // 3] * draws,
             u=np.full(2 * draws, 1 - 2.0 ** -24, np.float32), final=final, temps=[temperature] * draws,
             q=np.tile(np.stack([q, q]), (draws, 1)), held=np.tile(c["held"], (draws, 1)),
             logits=c["logits"].repeat(draws, 1))
    return c, picks


# A share is what is left of a probability less its rounding, some 2^-26 of it. The kernel's exponential is right to
# 2^-46, the row's sum of them too, and the oracle's to far more: the sum of the shares up to a token is off by
# at most 2^-45 of the probabilities up to there.
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("vocab,draws", [(700, 60), (5003, 60), (151667, 12)])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_a_draft_that_follows_the_model(vocab, draws, temperature, dtype):
    for seed in range(3):
        c, picks = follows(seed, vocab, dtype, draws, temperature)
        expected = want(c)
        assert [t[0] for t in expected[0]] == picks and expected[2] == [1] * draws
        same(call(c), expected)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("vocab", [151667, 1 << 20])
@pytest.mark.parametrize("tokens", [1, 2, 1 << 17])
def test_nothing_above_the_draft_in_a_large_row(tokens, vocab, dtype):
    # equal weights of a power of two of tokens, and a draft that equals them exactly; a number that is not below 1
    g = np.random.default_rng(tokens)
    place = np.sort(g.choice(vocab, tokens, replace=False))
    x = torch.full((2, vocab), -math.inf)
    x[:, place] = 1.5
    q = torch.zeros((2, vocab))
    q[:, place] = 1.0 / tokens
    for final in (0.0, 0.3, 0.5, 1 - 2.0 ** -24):
        t, p, n = scoring.verify_drafts(x.to(DT[dtype]).cuda(), cuda([0, int(place[0])]), cuda([0, 2], torch.int32), 2,
                                        cuda([0.0, 1.0]), cuda([final]), draft_probs=q.cuda())
        assert n.tolist() == [1] and t[0].tolist() == [place[int(final * tokens)], -1]


# The remainder is some 0.4 of the noise; the draft is within 2^-20 of the model for 0.8 2^-20 / noise of its mass.
# What the kernel leaves to the chord is below 2^-22 of that mass, 2^-36 with the noise of 2^-6, 2^-29 of the
# remainder: a random number is so near to one of 2^14.3 borders with a probability of 2^-14 (2^-20 with
# 2^-3; with 2^-10 the remainder is summed again, and 2^-45 of the row's sum is unknown).
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("noise", [2.0 ** -3, 2.0 ** -6, 2.0 ** -10])
@pytest.mark.parametrize("vocab,sequences", [(20003, 40), (20003, 1), (3001, 40)])
def test_drafts_close_to_the_model(vocab, sequences, noise, dtype):
    for seed in range(2):
        g = np.random.default_rng(seed)
        news = [2 + b % 3 for b in range(sequences)]
        c = make(seed + 60, news, vocab, dtype, probs=True, temps=list(g.choice([0.7, 1.0, 1.3], sequences)))
        for b, n in enumerate(news):
            t = float(np.float32(c["temps"][b]))
            for i in range(c["starts"][b], c["starts"][b] + n):
                p = O.weights(c["held"][i], t)
                p /= p.sum()
                q = p * np.exp(noise * g.standard_normal(vocab))
                c["q"][i] = (q / q.sum()).astype(np.float32)
                if i + 1 < c["starts"][b] + n:
                    # a token that the draft likes better, which is rejected, or one that it likes less
                    more = c["q"][i] > p * (1 + 2.0 ** -20)
                    c["ids"][i + 1] = int(g.choice(np.flatnonzero(more if g.random() < 0.6 else ~more)))
        c["u"][:] = 1 - 2.0 ** -24
        expected = want(c)
        assert sequences == 1 or 1 in expected[2] and max(expected[2]) > 1
        same(call(c), expected)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("vocab", [5003, 151667])
def test_every_token_of_a_large_row_rejected(vocab, dtype):
    # three tokens that can be, and siblings that name them all, with numbers that are not below 1: a draw from all
    place = [3, vocab // 2, vocab - 1]
    x = torch.full((4, vocab), -math.inf)
    x[:, place] = torch.tensor([1.0, 2.0, 0.5])
    starts, parents = cuda([0, 4], torch.int32), cuda([-1, 0, 0, 0], torch.int32)
    for last, final in ((1.0, 0.0), (1.0, 0.2), (1.0, 0.5), (1.0, 0.99), (0.5, 0.5)):
        u = cuda([0.0, 1.0, 1.0, last])
        t, p, n = scoring.verify_drafts(x.to(DT[dtype]).cuda(), cuda([0, *place]), starts, 4, u, cuda([final]), parents=parents)
        tokens, path = O.verify(x.numpy(), [0, *place], [-1, 0, 0, 0], u.tolist(), np.float32(final))
        assert t[0, :int(n)].tolist() == tokens and p[0, :int(n)].tolist() == path
        assert len(path) == (2 if last < 1 else 1)
