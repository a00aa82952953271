"""Verifies drafted trees of tokens with int4 weights and a paged 8-bit cache.

    python examples/verify_tree.py [--steps 8] [--cache e4m3|int8|16]

A small decoder with random weights (its products are ``torch.ops.w4a16.gemm``)
continues a few prompts of different lengths. Each step drafts a tree of
tokens per sequence and runs all trees through the model at once:

    qkv product -> kv_write (rotates q and k, quantises, stores)
                -> tree_attention (each token sees the cache and its ancestors)
                -> output product ... -> token_logprobs (what would come next)

Where the model's own choice is in the tree, it is accepted and the next one is
looked up in the same pass; accepted tokens' keys and values move to the end of
the sequence (kv_read, kv_write). The text is what one token at a time would
give. The draft here guesses from the model's previous alternatives.
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_only_int4_unpack_amd import attn, op, serve_op  # noqa: E402
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
    def __init__(self, s: Sizes, sequences: int, cache=torch.float8_e4m3fn, seed=0):
        self.s = s
        qkv = (s.q_heads + 2 * s.kv_heads) * s.head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((s.vocab, s.hidden), generator=g, device="cuda").to(s.dtype)
        self.qkv = [Linear(s.hidden, qkv, s.dtype, seed + 2 * i + 1) for i in range(s.layers)]
        self.out = [Linear(s.q_heads * s.head_dim, s.hidden, s.dtype, seed + 2 * i + 2)
                    for i in range(s.layers)]
        self.head = Linear(s.hidden, s.vocab, s.dtype, seed + 99)
        # one page table for all layers: sequence b holds pages b, b + sequences, ...
        self.caches = [attn.kv_cache(sequences * s.pages_each, s.kv_heads, s.head_dim, s.page,
                                     cache or s.dtype) for _ in range(s.layers)]
        self.table = attn.rope_table(s.pages_each * s.page, attn.rope_frequencies(s.head_dim))
        self.block_table = torch.arange(sequences * s.pages_each, dtype=torch.int32, device="cuda") \
            .view(s.pages_each, sequences).t().contiguous()

    def slots(self, sequence, places):
        """Cache slots of token places of a sequence (both int64 [tokens])."""
        page = self.block_table[sequence, places // self.s.page]
        return page.long() * self.s.page + places % self.s.page

    def __call__(self, tokens, sequence, places, positions, kv_lens, q_starts, max_q, mask=None):
        """Logits after each of `tokens`, whose keys and values go to `places`."""
        s = self.s
        slots = self.slots(sequence, places)
        x = self.embed[tokens]
        for qkv, out, cache in zip(self.qkv, self.out, self.caches):
            h = qkv(F.rms_norm(x, (s.hidden,)))
            q, k, v = h.view(len(tokens), -1, s.head_dim).split([s.q_heads, s.kv_heads, s.kv_heads], 1)
            q = serve_op.kv_write(k, v, slots, cache, positions, self.table, False, q)
            a, _ = serve_op.tree_attention(q, cache, self.block_table, kv_lens, q_starts, max_q, mask)
            x = x + out(a.view(len(tokens), -1))
        return self.head(F.rms_norm(x, (s.hidden,)))

    def move(self, sequence, places, to):
        """Cached tokens to other places of their sequences (rotated already)."""
        for cache in self.caches:
            k, v = serve_op.kv_read(cache, self.slots(sequence, places), self.s.dtype)
            serve_op.kv_write(k, v, self.slots(sequence, to), cache)


def ints(x, dtype=torch.int64):
    return torch.tensor(x, dtype=dtype, device="cuda")


def run(model, texts, cached, trees):
    """One pass: per sequence, `trees[b]` = (tokens, parents) after `cached[b]` cached ones.
    Returns log-probabilities' (alternatives, ids) per token and where sequences start."""
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
    logits = model(ints(tokens), ints(seq), ints(places), ints(pos),
                   ints([c + len(t[0]) for c, t in zip(cached, trees)], torch.int32),
                   ints(starts, torch.int32), max(len(t[0]) for t in trees),
                   None if plain else attn.tree_mask(parents))
    # the likelihood of each token's own choice, and the alternatives to draft from
    logprob, entropy, top, top_ids = serve_op.token_logprobs(logits, logits.argmax(-1), 4)
    return starts, logprob, top, top_ids


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


def generate(model, prompts, steps, drafts=True):
    """Greedy continuations. Returns texts, their chosen tokens' log-probabilities, passes."""
    texts = [list(p) for p in prompts]
    scores = [[] for _ in prompts]
    cached = [0] * len(prompts)
    seen: dict[int, list[int]] = {}                   # token -> what the model last put after it
    trees = [chain(p) for p in prompts]
    for _ in range(steps):
        starts, logprob, _, ids = run(model, texts, cached, trees)
        logprob, ids = logprob.tolist(), ids.tolist()
        seq, come, to = [], [], []
        for b, (toks, par) in enumerate(trees):
            at = starts[b]
            for j, t in enumerate(toks):
                seen[t] = ids[at + j]
            # the prompt's chain, or the root of a draft, is known; then follow the model
            node = len(toks) - 1 if cached[b] == 0 else 0
            path = list(range(node + 1))
            while True:
                best = ids[at + node][0]
                texts[b].append(best)
                scores[b].append(logprob[at + node])
                kids = [j for j in range(len(toks)) if par[j] == node and j > path[-1] and toks[j] == best]
                if not kids:
                    break
                node = kids[0]
                path.append(node)
            moved = [(i, j) for i, j in enumerate(path) if i != j]
            seq += [b] * len(moved)
            come += [cached[b] + j for _, j in moved]
            to += [cached[b] + i for i, _ in moved]
            cached[b] += len(path)
        if seq:
            model.move(ints(seq), ints(come), ints(to))
        trees = [draft(t[-1], lambda x: seen.get(x, [x]), *((3, 2) if drafts else (0, 0))) for t in texts]
    return texts, scores


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--cache", choices=sorted(CACHES), default="e4m3")
    a = p.parse_args(argv)
    g = torch.Generator().manual_seed(1)
    s = Sizes()
    # prompts that repeat, so that drafts from what came before are sometimes right
    prompts = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (100, 1, 37)]
    model = Decoder(s, len(prompts), CACHES[a.cache])
    texts, scores = generate(model, prompts, a.steps)
    for b, text in enumerate(texts):
        new = text[len(prompts[b]):]
        print(f"sequence {b}: {len(prompts[b])} tokens + {len(new)} in {a.steps} passes, "
              f"mean log-probability {sum(scores[b]) / len(new):.3f}: {new[:12]}", flush=True)


if __name__ == "__main__":
    main()
