"""Verifies drafted trees of tokens with int4 weights, adapters and a paged 8-bit cache.

    python examples/verify_tree.py [--steps 8] [--cache e4m3|int8|16] [--adapters 0]
                                   [--samples 1] [--temperature 0]

A small decoder with random weights (its products are ``torch.ops.w4a16.gemm``)
continues a few prompts of different lengths, each ``--samples`` times and with a
low-rank adapter of its own, or none. Each step drafts a tree of tokens per
sequence and runs all trees through the model at once:

    pages_resize (pages for the new tokens) and lora_plan, once a step
    qkv product -> lora (each sequence's adapter)
                -> kv_write (rotates q and k, quantises, stores)
                -> tree_attention (each token sees the cache and its ancestors)
                -> output product ... -> verify_drafts (what is accepted)
                -> kv_compact (accepted tokens' keys and values close up)

The prompts run once; ``pages_fork`` then lets the samples share their full pages.
The text is distributed as one token at a time would be; at temperature 0 it is
the model's own choice. The draft here guesses from the model's previous
alternatives.
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_only_int4_unpack_amd import attn, batch_op, op, paging, serve_op  # noqa: E402
from weight_only_int4_unpack_amd import w4a16 as W  # noqa: E402

GROUP = 128
CACHES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "16": None}


@dataclass
class Sizes:
    hidden: int = 1024
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    layers: int = 2
    vocab: int = 4096
    page: int = 16
    pages_each: int = 32
    rank: int = 16
    dtype: torch.dtype = torch.bfloat16


class Linear:
    """Random symmetric int4 weights of unit gain."""

    def __init__(self, k, n, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        q = torch.randint(0, 16, (k, n), generator=g, dtype=torch.uint8)
        self.b_q = torch.from_numpy(W.pack_int4(q.numpy())).cuda()
        self.scales = torch.full((k // GROUP, n), 1 / (4.6 * math.sqrt(k)), dtype=dtype, device="cuda")

    def __call__(self, x):
        return op.gemm(x, self.b_q, self.scales, None, GROUP)


class Decoder:
    """`adapters` of them belong to the qkv products; sequence b takes number b % (adapters + 1),
    the last of which is none, or, forked, that of the sequence it continues."""

    def __init__(self, s: Sizes, sequences: int, cache=torch.float8_e4m3fn, seed=0, adapters=0):
        self.s, self.adapters = s, adapters
        self.adapter = torch.arange(sequences, dtype=torch.int32, device="cuda") % (adapters + 1)
        qkv = (s.q_heads + 2 * s.kv_heads) * s.head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((s.vocab, s.hidden), generator=g, device="cuda").to(s.dtype)
        self.qkv = [Linear(s.hidden, qkv, s.dtype, seed + 2 * i + 1) for i in range(s.layers)]
        self.out = [Linear(s.q_heads * s.head_dim, s.hidden, s.dtype, seed + 2 * i + 2)
                    for i in range(s.layers)]
        self.head = Linear(s.hidden, s.vocab, s.dtype, seed + 99)
        down, up = (adapters, s.rank, s.hidden), (adapters, qkv, s.rank)
        self.lora = [[torch.randn(shape, generator=g, device="cuda").mul_(shape[2] ** -0.5).to(s.dtype)
                      for shape in (down, up)] for _ in range(s.layers)]
        # one pool of pages for all layers
        self.caches = [attn.kv_cache(sequences * s.pages_each, s.kv_heads, s.head_dim, s.page,
                                     cache or s.dtype) for _ in range(s.layers)]
        self.group = paging.cache_group(self.caches)
        self.pool = paging.page_pool(sequences * s.pages_each, sequences, s.pages_each, s.page)
        self.table = attn.rope_table(s.pages_each * s.page, attn.rope_frequencies(s.head_dim))

    def slots(self, sequence, places):
        """Cache slots of token places of a sequence (both int64 [tokens])."""
        page = self.pool.block_table[sequence, places // self.s.page]
        return page.long() * self.s.page + places % self.s.page

    def resize(self, lens):
        """Pages for `lens` tokens of the first sequences."""
        rows = range(len(lens))
        self.copy(rows, *batch_op.pages_resize(self.pool, ints(rows, torch.int32), lens))

    def fork(self, parents, children):
        """Continues sequences as others too."""
        self.adapter[ints(children)] = self.adapter[ints(parents)]
        self.copy(children, *batch_op.pages_fork(self.pool, ints(parents, torch.int32), ints(children, torch.int32)))

    def copy(self, rows, served, src, dst):
        """The pages that a change of `rows` has to copy. A sequence that was not served has no place for
        its tokens: nothing may run on it."""
        batch_op.kv_copy_pages(self.group, src, dst)
        if not served.all():
            short, free = [r for r, ok in zip(rows, served.tolist()) if not ok], int((self.pool.refs == 0).sum())
            raise RuntimeError(f"no room for sequences {short}: up to {self.s.pages_each * self.s.page} tokens each, "
                               f"{free} pages free")

    def __call__(self, tokens, sequence, places, positions, kv_lens, q_starts, max_q, mask=None):
        """Logits after each of `tokens`, whose keys and values go to `places`."""
        s = self.s
        slots = self.slots(sequence, places)
        rows = self.pool.block_table[:len(kv_lens)]
        plan = self.adapters and batch_op.lora_plan(self.adapter[sequence], self.adapters)
        x = self.embed[tokens]
        for qkv, lora, out, cache in zip(self.qkv, self.lora, self.out, self.caches):
            x1 = F.rms_norm(x, (s.hidden,))
            h = qkv(x1)
            if plan:
                h = batch_op.lora(x1, *lora, plan, base=h)
            q, k, v = h.view(len(tokens), -1, s.head_dim).split([s.q_heads, s.kv_heads, s.kv_heads], 1)
            q = serve_op.kv_write(k, v, slots, cache, positions, self.table, False, q)
            a, _ = serve_op.tree_attention(q, cache, rows, kv_lens, q_starts, max_q, mask)
            x = x + out(a.view(len(tokens), -1))
        return self.head(F.rms_norm(x, (s.hidden,)))


def ints(x, dtype=torch.int64):
    return torch.tensor(x, dtype=dtype, device="cuda")


@dataclass
class Pass:
    """What one run of all trees is made of: tokens and parents of all nodes, where sequences
    start among them (also as `q_starts`), cached lengths with them, and the logits."""
    tokens: torch.Tensor
    parents: torch.Tensor
    starts: list
    q_starts: torch.Tensor
    kv_lens: torch.Tensor
    max_q: int
    logits: torch.Tensor


def forward(model, cached, trees):
    """One pass: per sequence, `trees[b]` = (tokens, parents) after `cached[b]` cached ones."""
    tokens, seq, places, pos, starts, parents = [], [], [], [], [0], []
    for b, (toks, par) in enumerate(trees):
        depth = []
        for j, p in enumerate(par):
            depth.append(depth[p] + 1 if p >= 0 else 0)
            places.append(cached[b] + j)
        pos += [cached[b] + d for d in depth]
        tokens += toks
        seq += [b] * len(toks)
        starts.append(len(tokens))
        parents.append(par)
    plain = all(p == list(range(-1, len(p) - 1)) for p in parents)
    lens, max_q = ints([c + len(t[0]) for c, t in zip(cached, trees)], torch.int32), max(len(t[0]) for t in trees)
    model.resize(lens)
    tokens, q_starts = ints(tokens), ints(starts, torch.int32)
    logits = model(tokens, ints(seq), ints(places), ints(pos), lens, q_starts, max_q,
                   None if plain else attn.tree_mask(parents))
    return Pass(tokens, ints(sum(parents, []), torch.int32), starts, q_starts, lens, max_q, logits)


def run(model, texts, cached, trees):
    """One pass. Returns log-probabilities' (alternatives, ids) per token and where sequences start."""
    p = forward(model, cached, trees)
    # the likelihood of each token's own choice, and the alternatives to draft from
    logprob, entropy, top, top_ids = serve_op.token_logprobs(p.logits, p.logits.argmax(-1), 4)
    return p.starts, logprob, top, top_ids


def chain(tokens):
    return tokens, list(range(-1, len(tokens) - 1))


def draft(first, guesses, width=3, depth=2):
    """`first`, then a tree of guesses: at each of `depth` levels the best node gets `width`."""
    tokens, parents, node = [first], [-1], 0
    for level in range(depth):
        kids = guesses(tokens[node])[:width]
        parents += [node] * len(kids)
        node = len(tokens)
        tokens += kids
    return tokens, parents


def generate(model, prompts, steps, drafts=True, samples=1, temperature=0.0, seed=0):
    """Continuations of each prompt: sequence b is one of prompt b % len(prompts).
    Returns texts, their chosen tokens' log-probabilities."""
    P, rows = len(prompts), len(prompts) * samples
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda n: torch.rand(n, generator=g, device="cuda")                     # noqa: E731
    temperatures = torch.full((rows,), temperature, device="cuda")
    texts = [list(prompts[b % P]) for b in range(rows)]
    scores = [[] for _ in range(rows)]
    cached = [len(t) for t in texts]
    seen: dict[int, list[int]] = {}                   # token -> what the model last put after it
    model.resize(torch.zeros(rows, dtype=torch.int32, device="cuda"))
    for step in range(steps):
        if step == 0:
            # the prompts' chains, once each; a sequence's first token follows its prompt's last
            p = forward(model, [0] * P, [chain(t) for t in prompts])
            model.fork([b % P for b in range(P, rows)], list(range(P, rows)))
            at = [p.starts[b % P + 1] - 1 for b in range(rows)]
            root, q_starts = ints(at), ints(range(rows + 1), torch.int32)
            tokens, path, counts = batch_op.verify_drafts(p.logits[root], p.tokens[root], q_starts, 1, rand(rows),
                                                          rand(rows), None, None, temperatures)
        else:
            trees = [draft(t[-1], lambda x: seen.get(x, [x]), *((3, 2) if drafts else (0, 0))) for t in texts]
            p = forward(model, cached, trees)
            tokens, path, counts = batch_op.verify_drafts(p.logits, p.tokens, p.q_starts, p.max_q,
                                                          rand(len(p.tokens)), rand(rows), p.parents, None,
                                                          temperatures)
            cached = batch_op.kv_compact(model.group, model.pool.block_table[:rows], p.kv_lens, p.q_starts, path,
                                         counts)
            model.resize(cached)
            cached, at = cached.tolist(), p.starts
        # the alternatives to draft from, and the likelihood of what was chosen
        ids = serve_op.token_logprobs(p.logits, p.tokens, 4)[3].tolist()
        seen.update(zip(p.tokens.tolist(), ids))
        tokens, path, counts = tokens.tolist(), path.tolist(), counts.tolist()
        new = [t[:n] for t, n in zip(tokens, counts)]
        places = [at[b] + j for b in range(rows) for j in path[b][:counts[b]]]
        logprob = serve_op.token_logprobs(p.logits[ints(places)], ints(sum(new, [])))[0].tolist()
        for b in range(rows):
            texts[b] += new[b]
            scores[b] += logprob[:counts[b]]
            logprob = logprob[counts[b]:]
    return texts, scores


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--cache", choices=sorted(CACHES), default="e4m3")
    p.add_argument("--adapters", type=int, default=0)
    p.add_argument("--samples", type=int, default=1)
    p.add_argument("--temperature", type=float, default=0.0)
    a = p.parse_args(argv)
    g = torch.Generator().manual_seed(1)
    s = Sizes()
    # prompts that repeat, so that drafts from what came before are sometimes right
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (100, 1, 37)]
    model = Decoder(s, len(prompts) * a.samples, CACHES[a.cache], adapters=a.adapters)
    texts, scores = generate(model, prompts, a.steps, samples=a.samples, temperature=a.temperature)
    for b, text in enumerate(texts):
        prompt = len(prompts[b % len(prompts)])
        new = text[prompt:]
        print(f"sequence {b}: {prompt} tokens + {len(new)} in {a.steps} passes, "
              f"mean log-probability {sum(scores[b]) / len(new):.3f}: {new[:12]}", flush=True)


if __name__ == "__main__":
    main()
