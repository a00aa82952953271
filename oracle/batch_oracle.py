"""Plain fp64 oracle of the operators of a batch of requests (verification of drafts,
adapters, pages of the cache), on the CPU. Shares no code with the GPU library:
NumPy and Python lists, one sequence, token and page at a time.
"""
from __future__ import annotations

import numpy as np


def weights(x, temperature):
    """exp((x - max x) / temperature), or 1 at the first largest; None: no softmax."""
    x = np.asarray(x, np.float64)
    top = x.max()
    if not np.isfinite(top):
        return None
    if not temperature > 0:
        w = np.zeros_like(x)
        w[int(np.argmax(x))] = 1.0
        return w
    with np.errstate(invalid="ignore", over="ignore"):
        d = (x - top) / temperature
    return np.where(x == -np.inf, 0.0, np.exp(d))


def draw(r, border):
    """The first index at which the cumulative sum passes border of the whole."""
    up = np.cumsum(r)
    k = int(np.searchsorted(up, border * up[-1], side="right")) if border == border else len(r)
    return min(k, int(np.flatnonzero(r)[-1]))


def verify(logits, ids, parents, uniforms, final, probs=None, temperature=1.0):
    """One sequence: (tokens, path). parents[i] for i >= 1; probs[i]: of the token after node i."""
    n, V = len(ids), logits.shape[1]
    node, path, tokens = 0, [0], []
    while True:
        w = weights(logits[node], temperature)
        if w is None:
            return tokens + [-1], path
        total, removed, gone, found, drawn = w.sum(), 0.0, [], None, False
        for c in range(node + 1, n):
            if parents[c] != node:
                continue
            t = ids[c]
            known = 0 <= t < V
            if probs is not None:
                q = float(probs[node][t]) if known else 0.0
                if float(uniforms[c]) * q * total < (w[t] if known else 0.0):
                    found = c
                    break
                drawn = True
            elif known and t not in gone:
                if float(uniforms[c]) * (total - removed) < w[t]:
                    found = c
                    break
                gone.append(t)
                removed += w[t]
        if found is None:
            r = w.copy()
            if drawn and temperature > 0:
                q = np.asarray(probs[node], np.float64)
                with np.errstate(invalid="ignore"):
                    r = np.fmax(w / total - q, 0.0)
            elif gone:
                r[gone] = 0.0
            return tokens + [draw(r if r.any() else w, float(final))], path
        path.append(found)
        tokens.append(int(ids[found]))
        node = found


def lora(x, a, b, index, base=None, scales=None, ranks=None):
    """(out, bound parts): fp64 result, sum |v b|, and sum_r |b| sum_k |x a|, scaled."""
    x, a, b = (np.asarray(z, np.float64) for z in (x, a, b))
    T, N = len(x), b.shape[1]
    out = np.zeros((T, N)) if base is None else np.asarray(base, np.float64).copy()
    vb, deep = np.zeros((T, N)), np.zeros((T, N))
    for t, i in enumerate(index):
        if not 0 <= i < len(a):
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        s = 1.0 if scales is None else float(scales[i])
        v = a[i, :r] @ x[t]
        out[t] += s * (b[i, :, :r] @ v)
        vb[t] = abs(s) * (np.abs(b[i, :, :r]) @ np.abs(v))
        deep[t] = abs(s) * (np.abs(b[i, :, :r]) @ (np.abs(a[i, :r]) @ np.abs(x[t])))
    return out, vb, deep


class Pool:
    """A pool of pages as Python lists."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = list(refs), [list(r) for r in table], list(lens), page

    def _known(self, p):
        return 0 <= p < len(self.refs)

    def _release(self, p):
        if self._known(p) and self.refs[p] > 0:
            self.refs[p] -= 1

    def _pages(self, n):
        return -(-n // self.page)

    def resize(self, rows, lens):
        room = len(self.table[0]) * self.page if self.table else 0
        free = [p for p, r in enumerate(self.refs) if r == 0]
        start = list(self.refs)
        short, done, served, src, dst, gone = False, set(), [], [], [], []
        for r, n in zip(rows, lens):
            served.append(0)
            src.append(-1)
            dst.append(-1)
            first = r not in done
            done.add(r)
            if not (first and 0 <= r < len(self.lens) and 0 <= n <= room):
                continue
            old = min(max(self.lens[r], 0), room)
            kept = min(old, n)
            entry, need, own = self._pages(old), max(self._pages(n) - self._pages(old), 0), -1
            if kept % self.page:
                p = self.table[r][kept // self.page]
                if self._known(p) and start[p] > 1:
                    own, entry, need = p, kept // self.page, need + 1
            if need and (short or need > len(free)):
                short = True
                continue
            new = [free.pop(0) for _ in range(need)]
            for k, p in enumerate(new):
                self.table[r][entry + k] = p
                self.refs[p] = 1
            if own >= 0:
                src[-1], dst[-1] = own, new[0]
                gone.append(own)
            for k in range(self._pages(n), self._pages(old)):
                gone.append(self.table[r][k])
                self.table[r][k] = -1
            self.lens[r] = n
            served[-1] = 1
        for p in gone:
            self._release(p)
        return served, src, dst

    def fork(self, parents, children):
        room = len(self.table[0]) * self.page if self.table else 0
        free = [p for p, r in enumerate(self.refs) if r == 0]
        lens, table = list(self.lens), [list(r) for r in self.table]
        short, done, served, src, dst = False, set(), [], [], []
        for a, c in zip(parents, children):
            served.append(0)
            src.append(-1)
            dst.append(-1)
            first = c not in done
            done.add(c)
            rows = len(lens)
            if not (first and 0 <= c < rows and 0 <= a < rows and a != c and lens[c] <= 0):
                continue
            n = min(max(lens[a], 0), room)
            full, part = n // self.page, n % self.page > 0
            if part and (short or not free):
                short = True
                continue
            for k in range(full):
                p = table[a][k]
                self.table[c][k] = p
                if self._known(p):
                    self.refs[p] += 1
            if part:
                p = free.pop(0)
                self.table[c][full] = p
                self.refs[p] = 1
                dst[-1] = p
                src[-1] = table[a][full] if self._known(table[a][full]) else -1
            self.lens[c] = n
            served[-1] = 1
        return served, src, dst


def compact(n, path, count):
    """Which of a sequence's new tokens stay: [(from, to)] places among them."""
    moves, above = [], -1
    for j in range(max(count, 0)):
        if j >= len(path) or not above < path[j] < n:
            break
        moves.append((int(path[j]), j))
        above = path[j]
    return moves
