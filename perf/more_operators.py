"""Cases of the operators of a serving step for many users: verification of drafted tokens from given random
numbers, low-rank adapters beside a shared product, forks of paged sequences with the copies of their pages,
and compaction of the accepted tokens in the cache.

``run`` computes an operator in its plain form (elementary torch operations) or, where ``own`` is true, by the
calls a user makes of ``weight_only_int4_unpack_amd``. ``exact`` is the operator's definition in fp64, written
apart from the plain form.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # a single user's draft of 4 tokens, a small vocabulary, with the draft model's probabilities: latency
        dict(name="verify-one", op="verify", dtype="bf16", batch=1, new=5, vocab=32000, tree=False, probs=True,
             greedy=False, ragged=False),
        # a full batch, 64 sequences with up to 5 drafted tokens each over a large odd vocabulary
        dict(name="verify-chains", op="verify", dtype="bf16", batch=64, new=6, vocab=151667, tree=False, probs=True,
             greedy=False, ragged=True),
        # 16 trees of up to 24 tokens, as the attention case of that size; some users greedy, most not
        dict(name="verify-trees", op="verify", dtype="bf16", batch=16, new=24, vocab=151667, tree=True, probs=False,
             greedy=True, ragged=True),
        # one token of one user with a small adapter beside a square projection: latency
        dict(name="lora-one", op="lora", dtype="fp16", tokens=1, each=1, adapters=4, rank=8, k=4096, n=4096, mixed=False),
        # a decode batch, 64 users with 32 adapters (some users without) beside the widest projection
        dict(name="lora-decode", op="lora", dtype="bf16", tokens=64, each=1, adapters=32, rank=16, k=5120, n=17408,
             mixed=False),
        # 16 drafted trees of 24 tokens, adapters of different ranks up to 64, an odd inner size
        dict(name="lora-trees", op="lora", dtype="fp16", tokens=384, each=24, adapters=8, rank=64, k=2112, n=5120,
             mixed=True),
        # prompts of 4 users, 2048 tokens each, rank 64: read and written once, bound by HBM
        dict(name="lora-prompts", op="lora", dtype="bf16", tokens=8192, each=2048, adapters=4, rank=64, k=5120, n=17408,
             mixed=False),
        # one sequence continued in 3 ways after a shared prompt, a small model
        dict(name="fork-few", op="fork", fmt="e4m3", parents=1, each=3, tokens=1000, layers=8, heads=8, dim=128, page=16),
        # a step of a wide search, 10 sequences with 4 continuations each, large 16-bit pages
        dict(name="fork-many", op="fork", fmt="bf16", parents=10, each=4, tokens=900, layers=16, heads=8, dim=128, page=64),
        # the accepted tokens of one tree moved to the sequence's end
        dict(name="compact-few", op="compact", fmt="bf16", batch=1, new=8, accepted=3, tokens=500, layers=8, heads=8,
             dim=128, page=16),
        # a batch of 64 trees of 24, up to 5 accepted each, all 32 layers of an e4m3 cache
        dict(name="compact-many", op="compact", fmt="e4m3", batch=64, new=24, accepted=5, tokens=500, layers=32, heads=8,
             dim=128, page=16),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    while True:
        c = _draw(rng)
        tops = [work(x) for x in listed() if x["op"] == c["op"]]
        w = work(c)
        if w["bytes"] <= max(t["bytes"] for t in tops) and w["flops"] <= max(t["flops"] for t in tops) \
                and _held(c) <= max(_held(x) for x in listed()):
            return c


def _draw(rng):
    op = rng.choice(["verify", "verify", "lora", "lora", "fork", "compact"])
    c = dict(op=op)
    if op == "verify":
        tree = rng.choice([False, True])
        c.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), batch=_log_int(rng, 1, 128),
                 new=_log_int(rng, 1, 64 if tree else 12), vocab=_log_int(rng, 1000, 200000), tree=tree,
                 probs=not tree and rng.choice([False, True]), greedy=rng.choice([False, True]),
                 ragged=rng.choice([False, True]))
    elif op == "lora":
        each = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 2, 4096)])
        c.update(dtype=rng.choice(["bf16", "fp16"]), tokens=each * _log_int(rng, 1, 128), each=each,
                 adapters=_log_int(rng, 1, 64), rank=rng.choice([8, 16, 16, 24, 32, 64, 64, 128]),
                 k=8 * _log_int(rng, 32, 2176), n=8 * _log_int(rng, 32, 2176), mixed=rng.choice([False, True]))
    else:
        c.update(fmt=rng.choice(["bf16", "fp16", "e4m3"]))
        sizes = dict(tokens=_log_int(rng, 8, 2000), layers=_log_int(rng, 1, 32), heads=rng.choice([1, 2, 4, 5, 8]),
                     dim=rng.choice([64, 80, 96, 128, 128, 256]), page=rng.choice([16, 16, 32, 64, 128]))
        if op == "fork":
            c.update(parents=_log_int(rng, 1, 32), each=rng.choice([1, 2, 3, 4, 5]), **sizes)
        else:
            new = _log_int(rng, 2, 64)
            c.update(batch=_log_int(rng, 1, 128), new=new, accepted=rng.randint(1, min(8, (new + 1) // 2)), **sizes)
    return c


# ---------------------------------------------------------------- what a case is made of
def _news(case):
    """New tokens of each sequence of a batch: by the case alone."""
    if not case.get("ragged"):
        return [case["new"]] * case["batch"]
    return [max(1, case["new"] - (b * 5) % (case["new"] // 2 + 1)) for b in range(case["batch"])]


def _lens(case):
    """Cached tokens of each sequence, the new ones included: by the case alone."""
    count = case["parents"] if case["op"] == "fork" else case["batch"]
    least = case.get("new", 1)
    return [max(least, int(case["tokens"] * (1.0 - (0.5 * b * 0.6180339887) % 0.5))) for b in range(count)]


def _pages(case):
    """Pages of a cache case: those in use, those of continuations, and a few more."""
    lens, p = _lens(case), case["page"]
    used = sum(-(-n // p) for n in lens)
    return used + (len(lens) * case["each"] * (1 + -(-max(lens) // p)) // 2 + 2 if case["op"] == "fork" else 3)


def _token_bytes(case):
    """Of one token and head, key and value."""
    return 2 * (case["dim"] + 4 if case["fmt"] == "e4m3" else case["dim"] * 2)


def _held(case):
    """Bytes of a prepared case, roughly."""
    if case["op"] in ("fork", "compact"):
        return _pages(case) * case["page"] * case["layers"] * case["heads"] * _token_bytes(case)
    return work(case)["bytes"]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _starts(news):
    at = [0]
    for n in news:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    if case["op"] == "verify":
        _prepare_verify(s, g, random.Random(seed))
    elif case["op"] == "lora":
        _prepare_lora(s, g, random.Random(seed))
    else:
        _prepare_pages(s, g, random.Random(seed))
    if own:
        # what a program keeps: the order of a step's tokens by adapter, the layers' caches as one group
        from weight_only_int4_unpack_amd import adapters, attn, paging
        if case["op"] == "lora":
            s["plan"] = adapters.lora_plan(s["index"], case["adapters"])
        if case["op"] in ("fork", "compact"):
            s["group"] = paging.cache_group([attn.KVCache(*(None if x is None else x[i] for x in s["cache"]))
                                             for i in range(case["layers"])])
        if case["op"] == "fork":
            s["pool"] = paging.PagePool(s["refs"], s["table"], s["lens"], case["page"])
    return s


def _prepare_verify(s, g, rng):
    news, V = _news(s), s["vocab"]
    T = sum(news)
    x = torch.randn((T, V), generator=g, device="cuda") * 3
    # a few favourites a row, the first of them with some 0.8 of the probability
    liked = torch.randint(0, V, (T, 6), generator=g, device="cuda")
    x.scatter_(1, liked, math.log(V) + 7.0 - 1.5 * torch.arange(6, device="cuda")
               + torch.randn((T, 6), generator=g, device="cuda"))
    s["logits"] = x.to(DTYPES[s["dtype"]])
    s["q_starts"], s["max_q"] = _starts(news), max(news)
    parents, rank = [], []
    for n in news:
        tree = [-1]
        for i in range(1, n):
            # breadth first: a node's children follow each other, early nodes have more
            tree.append(rng.randint(max(tree[-1], 0), min(i - 1, max(tree[-1], 0) + 1)) if s["tree"] else i - 1)
        parents += tree
        rank += [sum(tree[j] == tree[i] for j in range(i)) for i in range(n)]
    s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda") if s["tree"] else None
    base = torch.repeat_interleave(s["q_starts"][:-1].long(), torch.tensor(news, device="cuda"), output_size=T)
    above = (base + torch.tensor(parents, device="cuda")).clamp(min=0)
    # the draft: the model's own logits with some noise, drawn from (chains) or its likeliest (trees)
    near = x + torch.randn((T, V), generator=g, device="cuda")
    s["probs_rows"] = torch.softmax(near, dim=-1) if s["probs"] else None
    if s["tree"]:
        near += torch.randn((T, V), generator=g, device="cuda")
        best = near.topk(max(rank) + 1, dim=-1).indices
        s["ids"] = best[above, torch.tensor(rank, device="cuda")]
    else:
        noise = torch.rand((T, V), generator=g, device="cuda").clamp_(min=1e-30).log_().neg_().log_()
        s["ids"] = (near - noise).argmax(-1)[above]
    s["uniforms"] = torch.rand((T,), generator=g, device="cuda")
    s["final"] = torch.rand((len(news),), generator=g, device="cuda")
    t = torch.rand((len(news),), generator=g, device="cuda") * 0.8 + 0.4
    if s["greedy"]:
        t[::3] = 0.0
    s["temperatures"] = t


def _prepare_lora(s, g, rng):
    dt, K, N, R, r = DTYPES[s["dtype"]], s["k"], s["n"], s["adapters"], s["rank"]
    T = s["tokens"]
    s["x"] = torch.randn((T, K), generator=g, device="cuda").to(dt)
    s["base"] = torch.randn((T, N), generator=g, device="cuda").to(dt)
    s["a"] = (torch.randn((R, r, K), generator=g, device="cuda") / math.sqrt(K)).to(dt)
    s["b"] = (torch.randn((R, N, r), generator=g, device="cuda") / math.sqrt(r)).to(dt)
    # one adapter a user, about an eighth of the users of a larger batch without one
    users = -(-T // s["each"])
    pick = [rng.randrange(R) if users < 8 or rng.random() > 0.125 else -1 for _ in range(users)]
    s["index"] = torch.tensor(pick, dtype=torch.int32, device="cuda").repeat_interleave(s["each"])[:T].contiguous()
    s["scales"] = torch.rand((R,), generator=g, device="cuda") + 0.5
    s["ranks"] = None
    if s["mixed"]:
        s["ranks"] = torch.tensor([max(1, r - (i * 5) % r) for i in range(R)], dtype=torch.int32, device="cuda")


def _prepare_pages(s, g, rng):
    lens, page, pages = _lens(s), s["page"], _pages(s)
    shape = (s["layers"], pages, s["heads"], page, s["dim"])
    if s["fmt"] == "e4m3":
        codes = [torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        for c in codes:
            for i in range(s["layers"]):
                c[i] = (torch.randn(shape[1:], generator=g, device="cuda") * 100).clamp_(-448, 448).to(c.dtype)
        s["cache"] = codes + [torch.rand(shape[:4], generator=g, device="cuda") * 0.01 for _ in range(2)]
    else:
        s["cache"] = [torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[s["fmt"]]) for _ in range(2)]
        s["cache"] += [None, None]
    order = list(range(pages))
    rng.shuffle(order)
    need = [-(-n // page) for n in lens]
    rows = []
    for n in need:
        rows.append(order[:n])
        del order[:n]
    if s["op"] == "fork":
        # row 0.. the sequences, then their continuations, which hold what an earlier step left them:
        # the first half of their sequence's pages, and one page of their own
        count, each = s["parents"], s["each"]
        refs = [0] * pages
        for row in rows:
            for p in row:
                refs[p] = 1
        for c in range(count * each):
            kept = rows[c % count][:need[c % count] // 2] + [order.pop()]
            for p in kept:
                refs[p] += 1
            rows.append(kept)
            lens.append(len(kept) * page - rng.randrange(page))
        s["refs"] = torch.tensor(refs, dtype=torch.int32, device="cuda")
        s["pairs"] = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                      ([c % count for c in range(count * each)], [count + c for c in range(count * each)])]
        s["none"] = torch.zeros(count * each, dtype=torch.int32, device="cuda")
    else:
        # a path's nodes lie behind the places they move to, or are there already
        news = _news(s)
        s["q_starts"] = _starts(news)
        path = torch.full((len(news), max(news)), -1, dtype=torch.int32)
        counts = []
        for b, n in enumerate(news):
            take = 1 + (b + s["accepted"] - 1) % s["accepted"] if len(news) > 1 else s["accepted"]
            ahead = rng.randint(0, 1)
            nodes = list(range(1 + ahead)) + sorted(rng.sample(range(take + 1, n), max(0, min(take - ahead, n - take - 1))))
            path[b, :len(nodes)] = torch.tensor(nodes)
            counts.append(len(nodes))
        s["path"] = path.cuda()
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    table = torch.full((len(rows), max(map(len, rows)) + 1), -1, dtype=torch.int32)
    for i, row in enumerate(rows):
        table[i, :len(row)] = torch.tensor(row)
    s["table"] = table.cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    return {"verify": _verify_plain, "lora": _lora_plain, "fork": _fork_plain, "compact": _compact_plain}[state["op"]](state)


def _run_own(s):
    from weight_only_int4_unpack_amd import adapters, paging, scoring
    if s["op"] == "verify":
        return scoring.verify_drafts(s["logits"], s["ids"], s["q_starts"], s["max_q"], s["uniforms"], s["final"],
                                     parents=s["parents"], draft_probs=s["probs_rows"], temperatures=s["temperatures"])
    if s["op"] == "lora":
        return adapters.lora(s["x"], s["a"], s["b"], s["plan"], base=s["base"], scales=s["scales"], ranks=s["ranks"])
    if s["op"] == "fork":
        pool, (parents, children) = s["pool"], s["pairs"]
        paging.pages_resize(pool, children, s["none"])
        served, src, dst = paging.pages_fork(pool, parents, children)
        paging.kv_copy_pages(s["group"], src, dst)
        return [served, src, dst, s["refs"], s["table"], s["lens"]] + _held_values(s)
    lens = paging.kv_compact(s["group"], s["table"], s["lens"], s["q_starts"], s["path"], s["counts"])
    return [lens] + _held_values(s)


def _held_values(s):
    """The cache's own buffers."""
    return [x for x in s["cache"] if x is not None]


def _weights(x, temperature):
    """exp((x - max x) / temperature) in 64 bits; 1 at the first largest where the temperature is 0."""
    x = x.double()
    top = x.amax(-1, keepdim=True)
    t = temperature.double()[..., None]
    at = torch.arange(x.shape[-1], device=x.device)
    hot = at == torch.where(x == top, at, x.shape[-1]).amin(-1, keepdim=True)
    return torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)), hot.double())


def _verify_plain(s):
    starts = s["q_starts"].long()
    n = starts[1:] - starts[:-1]
    T, V = s["logits"].shape
    B, most = n.shape[0], s["max_q"]
    dev = starts.device
    i = torch.arange(most, device=dev)
    rows = (starts[:-1, None] + i).clamp(max=T - 1)
    live = i < n[:, None]
    parent = i.expand(B, most) - 1 if s["parents"] is None else s["parents"].long()[rows]
    parent = torch.where(live & (i > 0), parent, -1)
    above = (starts[:-1, None] + parent).clamp(min=0)                       # row of logits that judges a node
    w = _weights(s["logits"], s["temperatures"][torch.searchsorted(starts, torch.arange(T, device=dev), right=True) - 1])
    total = w.sum(-1)
    ids = s["ids"][rows]
    mine = w[above, ids]
    u = s["uniforms"].double()[rows]
    sibling = (parent[:, :, None] == parent[:, None, :]) & (parent[:, :, None] >= 0) & (i[None, :] < i[:, None])
    if s["probs_rows"] is not None:
        passes = u * s["probs_rows"][above, ids].double() * total[above] < mine
    else:
        again = (sibling & (ids[:, :, None] == ids[:, None, :])).any(-1)     # a token that a sibling had before
        removed = (sibling * torch.where(again, 0.0, mine)[:, None, :]).sum(-1)
        passes = (u * (total[above] - removed) < mine) & ~again
    passes = passes & (parent >= 0)
    chosen = passes & ~(sibling & passes[:, None, :]).any(-1)
    # nodes whose ancestors are all chosen: the step relation, squared until it holds every depth
    step = (chosen[:, :, None] & (parent[:, :, None] == i)).float() + torch.eye(most, device=dev)
    for _ in range(max(1, (most - 1).bit_length())):
        step = torch.matmul(step, step).clamp(max=1.0)
    on = (step[:, :, 0] > 0) & live
    counts = on.sum(-1)
    path = torch.where(on, i, most).sort(-1).values
    path = torch.where(path < most, path, -1)
    last = torch.take_along_dim(path, (counts - 1).clamp(min=0)[:, None], 1)
    row = (starts[:-1, None] + last).squeeze(1)
    rest = w[row]
    below = parent == last                                                  # rejected children of the last node
    if s["probs_rows"] is not None:
        over = (rest / total[row][:, None] - s["probs_rows"][row].double()).clamp(min=0)
        left = torch.where(below.any(-1, keepdim=True), over, rest)
    else:
        gone = torch.zeros((B, V + 1), dtype=torch.bool, device=dev)
        gone.scatter_(1, torch.where(below, ids, V), True)
        left = torch.where(gone[:, :V], 0.0, rest)
    left = torch.where((left > 0).any(-1, keepdim=True), left, rest)
    upto = left.cumsum(-1)
    drawn = (upto <= s["final"].double()[:, None] * upto[:, -1:]).sum(-1)
    drawn = torch.minimum(drawn, (left > 0).long().mul(torch.arange(V, device=dev)).amax(-1))
    after = torch.take_along_dim(ids, torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0), 1)
    tokens = torch.where(i < counts[:, None] - 1, after, torch.where(i == counts[:, None] - 1, drawn[:, None], -1))
    return tokens, path.to(torch.int32), counts.to(torch.int32)


def _lora_plain(s):
    T, (R, r, K), N = s["x"].shape[0], s["a"].shape, s["b"].shape[1]
    dev = s["x"].device
    mine = s["index"][:, None] == torch.arange(R, device=dev)
    down = torch.matmul(s["x"].float(), s["a"].float().reshape(R * r, K).t()).reshape(T, R, r)
    keep = mine[:, :, None] * s["scales"][:, None]
    if s["ranks"] is not None:
        keep = keep * (torch.arange(r, device=dev) < s["ranks"][:, None])
    up = s["b"].float().transpose(1, 2).reshape(R * r, N)
    return (s["base"].float() + torch.matmul((down * keep).reshape(T, R * r), up)).to(s["x"].dtype)


def _fork_plain(s):
    refs, table, lens, page = s["refs"], s["table"], s["lens"], s["page"]
    parents, children = (x.long() for x in s["pairs"])
    entry = torch.arange(table.shape[1], device=table.device)
    # the continuations give their pages back
    held = entry < -(-lens[children] // page)[:, None]
    old = torch.where(held, table[children], 0).long()
    refs.scatter_add_(0, old.flatten(), -held.flatten().to(torch.int32))
    table[children] = torch.where(held, -1, table[children])
    # and share their sequence's full ones; a partly filled last page is copied to the lowest free one
    full = lens[parents] // page
    part = lens[parents] % page > 0
    free = torch.sort((refs != 0).to(torch.int32), stable=True).indices
    nth = part.long().cumsum(0) - 1
    ok = ~part | (nth < (refs == 0).sum())
    new = free[nth.clamp(0, refs.shape[0] - 1)].to(torch.int32)
    shared = (entry < full[:, None]) & ok[:, None]
    tail = (entry == full[:, None]) & (part & ok)[:, None]
    src = torch.where(part & ok, table[parents, full.long().clamp(max=table.shape[1] - 1)], -1)
    dst = torch.where(part & ok, new, -1)
    table[children] = torch.where(shared, table[parents], torch.where(tail, new[:, None], table[children]))
    refs.scatter_add_(0, torch.where(shared, table[parents], 0).long().flatten(), shared.flatten().to(torch.int32))
    refs.scatter_add_(0, torch.where(part & ok, new, 0).long(), (part & ok).to(torch.int32))
    lens[children] = torch.where(ok, lens[parents], 0)
    # where there is nothing to copy, a page in use is written over with itself
    same = table[parents, 0]
    at, to = torch.where(part & ok, src, same).long(), torch.where(part & ok, dst, same).long()
    for x in _held_values(s):
        y = x.view(torch.uint8) if x.element_size() == 1 else x
        y[:, to] = y[:, at]
    return [ok.to(torch.int32), src, dst, refs, table, lens] + _held_values(s)


def _compact_plain(s):
    table, lens, page = s["table"].long(), s["lens"].long(), s["page"]
    starts = s["q_starts"].long()
    n = starts[1:] - starts[:-1]
    first = lens - n
    j = torch.arange(s["path"].shape[1], device=table.device)
    kept = j < s["counts"][:, None]
    come = (first[:, None] + torch.where(kept, s["path"].long(), 0)).flatten()
    go = (first[:, None] + torch.where(kept, j, 0)).flatten()
    b = torch.arange(len(n), device=table.device).repeat_interleave(j.shape[0])
    p0, o0, p1, o1 = table[b, come // page], come % page, table[b, go // page], go % page
    for x in _held_values(s):
        y = x.view(torch.uint8) if x.element_size() == 1 else x
        y[:, p1, :, o1] = y[:, p0, :, o0]
    return [(first + s["counts"]).to(torch.int32)] + _held_values(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "verify":
        T, V, B = sum(_news(case)), case["vocab"], case["batch"]
        size = 4 if case["dtype"] == "fp32" else 2
        # every row once; with the draft's probabilities also the row where a chain stops
        return {"bytes": T * (V * size + 20) + B * (V * 4 * case["probs"] + 16 + 12 * case["new"]), "flops": 20 * T * V}
    if case["op"] == "lora":
        T, K, N, r = case["tokens"], case["k"], case["n"], case["rank"]
        used = min(case["adapters"], -(-T // case["each"]))
        return {"bytes": 2 * T * (K + 2 * N) + 2 * used * r * (K + N) + 4 * T, "flops": 2 * T * r * (K + N)}
    token = case["heads"] * _token_bytes(case) * case["layers"]
    lens = _lens(case)
    if case["op"] == "fork":
        copies = sum(n % case["page"] > 0 for n in lens) * case["each"]
        return {"bytes": copies * 2 * case["page"] * token + len(lens) * case["each"] * 4 * max(lens) // case["page"],
                "flops": 0}
    # about a quarter of a path is in its place already
    moved = sum(1 + (b + case["accepted"] - 1) % case["accepted"] if len(lens) > 1 else case["accepted"]
                for b in range(len(lens)))
    return {"bytes": int(1.5 * moved * token) + 4 * len(lens) * (case["new"] + 4), "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "lora": _exact_lora, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)


def _exact_verify(s):
    starts, most = s["q_starts"].tolist(), s["max_q"]
    ids, us, finals, temps = (s[k].tolist() for k in ("ids", "uniforms", "final", "temperatures"))
    out = [[], [], []]
    for b, t in enumerate(temps):
        lo, n = starts[b], starts[b + 1] - starts[b]
        over = list(range(-1, n - 1)) if s["parents"] is None else s["parents"][lo:lo + n].tolist()
        node, path, emitted = 0, [0], []
        while True:
            x = s["logits"][lo + node].double()
            if t > 0:
                p = torch.softmax(x / t, dim=0)
            else:
                p = torch.zeros_like(x)
                p[int(torch.nonzero(x == x.max())[0])] = 1.0
            kids = [c for c in range(node + 1, n) if over[c] == node]
            found, rest = None, p.clone()
            for c in kids:
                token = ids[lo + c]
                if s["probs_rows"] is not None:
                    q = s["probs_rows"][lo + node].double()
                    if us[lo + c] * float(q[token]) < float(p[token]):
                        found = c
                        break
                    rest = torch.relu(p - q)
                else:
                    here = float(rest[token])
                    if us[lo + c] * float(rest.sum()) < here:
                        found = c
                        break
                    rest[token] = 0.0
            if found is None:
                if not bool((rest > 0).any()):
                    rest = p
                up = torch.cumsum(rest, 0)
                k = int(torch.searchsorted(up, up[-1] * finals[b], right=True))
                emitted.append(min(k, int(torch.nonzero(rest)[-1])))
                break
            emitted.append(ids[lo + found])
            path.append(found)
            node = found
        fill = [-1] * (most - len(path))
        for o, v in zip(out, (emitted + fill, path + fill, len(path))):
            o.append(v)
    dev = s["logits"].device
    return (torch.tensor(out[0], device=dev), torch.tensor(out[1], dtype=torch.int32, device=dev),
            torch.tensor(out[2], dtype=torch.int32, device=dev))


def _exact_lora(s):
    y = s["base"].double()
    index = s["index"].tolist()
    for i in set(index) - {-1}:
        rows = torch.tensor([t for t, j in enumerate(index) if j == i], device=y.device)
        r = s["rank"] if s["ranks"] is None else int(s["ranks"][i])
        v = s["x"][rows].double() @ s["a"][i, :r].double().T
        y[rows] += float(s["scales"][i]) * (v @ s["b"][i, :, :r].double().T)
    return y


def _exact_fork(s):
    refs, table, lens, page = s["refs"].tolist(), s["table"].tolist(), s["lens"].tolist(), s["page"]
    pairs = list(zip(*(x.tolist() for x in s["pairs"])))
    for _, c in pairs:
        for k in range(-(-lens[c] // page)):
            refs[table[c][k]] -= 1
            table[c][k] = -1
        lens[c] = 0
    free = [p for p, r in enumerate(refs) if r == 0]
    src, dst = [], []
    for a, c in pairs:
        full = lens[a] // page
        for k in range(full):
            table[c][k] = table[a][k]
            refs[table[a][k]] += 1
        if lens[a] % page:
            table[c][full] = free.pop(0)
            refs[table[c][full]] = 1
            src.append(table[a][full])
            dst.append(table[c][full])
        else:
            src.append(-1)
            dst.append(-1)
        lens[c] = lens[a]
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1] * len(pairs), src, dst, refs, table, lens)]
    outs = []
    for x in _held_values(s):
        y = x.double()
        for p, q in zip(src, dst):
            if p >= 0:
                y[:, q] = y[:, p]
        outs.append(y)
    return ints + outs


def _exact_compact(s):
    table, lens, page = s["table"].tolist(), s["lens"].tolist(), s["page"]
    starts, path, counts = s["q_starts"].tolist(), s["path"].tolist(), s["counts"].tolist()
    outs = [x.double() for x in _held_values(s)]
    new = []
    for b, length in enumerate(lens):
        first = length - (starts[b + 1] - starts[b])
        for j in range(counts[b]):
            come, go = first + path[b][j], first + j
            if come != go:
                for y in outs:
                    y[:, table[b][go // page], :, go % page] = y[:, table[b][come // page], :, come % page]
        new.append(first + counts[b])
    return [torch.tensor(new, dtype=torch.int32, device="cuda")] + outs
