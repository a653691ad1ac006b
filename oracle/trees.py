"""Plain CPU oracle of drafted trees over a cache of pages: the pages' state moved on request by request, rotary
positions with several axes, attention by a table of who sees whom, acceptance along a tree.

Test infrastructure only, like the rest of this package. Written from the definitions in include/vc.h, in float64 and
Python's whole numbers.
"""
from __future__ import annotations

import numpy as np


class Pages:
    """The state of a pool, and K and V as arrays [n_pages][Hkv][page][d] of any type. `faults` counts what would be
    reported as VC_DEV_PAGES."""

    def __init__(self, n_pages, page, n_seq, max_pages, k=None, v=None):
        self.page, self.max_pages = page, max_pages
        self.refs = np.zeros(n_pages, np.int32)
        self.free = np.arange(n_pages - 1, -1, -1, dtype=np.int32)
        self.n_free = n_pages
        self.table = np.zeros((n_seq, max_pages), np.int32)
        self.len, self.held, self.next = (np.zeros(n_seq, np.int32) for _ in range(3))
        self.k, self.v = k, v
        self.faults = 0

    def _take(self):
        self.n_free -= 1
        p = int(self.free[self.n_free])
        self.refs[p] = 1
        return p

    def reserve(self, reqs):
        for seq, rows in reqs:
            n, held = int(self.len[seq]), int(self.held[seq])
            want = -(-(n + rows) // self.page)
            tail, inside = n // self.page, n % self.page
            copy = rows > 0 and inside > 0 and self.refs[self.table[seq, tail]] > 1
            if want > self.max_pages or max(0, want - held) + copy > self.n_free:
                self.faults += 1
                continue
            if copy:
                old, new = int(self.table[seq, tail]), self._take()
                self.refs[old] -= 1
                self.table[seq, tail] = new
                for x in (self.k, self.v):
                    if x is not None:
                        x[new, :, :inside] = x[old, :, :inside]
            while self.held[seq] < want:
                self.table[seq, self.held[seq]] = self._take()
                self.held[seq] += 1

    def fork(self, pairs):
        for src, dst in pairs:
            if self.held[dst]:
                self.faults += 1
                continue
            n = -(-int(self.len[src]) // self.page)
            self.table[dst, :n] = self.table[src, :n]
            self.refs[self.table[src, :n]] += 1
            self.held[dst], self.len[dst], self.next[dst] = n, self.len[src], self.next[src]

    def trim(self, reqs):
        for seq, rows, nxt in reqs:
            if rows < self.len[seq]:
                self.len[seq], self.next[seq] = rows, nxt
            keep = -(-int(self.len[seq]) // self.page)
            while self.held[seq] > keep:
                self.held[seq] -= 1
                p = int(self.table[seq, self.held[seq]])
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    self.free[self.n_free] = p
                    self.n_free += 1

    def compact(self):
        used = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        U = len(used)
        holes = [p for p in range(U) if self.refs[p] == 0]
        to = dict(zip([p for p in used if p >= U], holes))
        for src, dst in to.items():
            self.refs[dst], self.refs[src] = self.refs[src], 0
            for x in (self.k, self.v):
                if x is not None:
                    x[dst] = x[src]
        for seq in range(len(self.held)):
            for j in range(self.held[seq]):
                self.table[seq, j] = to.get(int(self.table[seq, j]), self.table[seq, j])
        self.n_free = len(self.refs) - U
        self.free[: self.n_free] = np.arange(len(self.refs) - 1, U - 1, -1)

    def commit(self, reqs):
        """reqs: (seq, rows, path or None, n_acc or None, advance). A sequence whose rows are not all its own is left."""
        for seq, rows, path, n_acc, advance in reqs:
            n = int(self.len[seq])
            if rows == 0:
                continue
            if not self.own(seq, rows):
                self.faults += 1
                continue
            m = rows if n_acc is None else min(max(int(n_acc), 0), rows)
            if path is not None:
                for i in range(m):
                    if not i <= path[i] < rows:
                        self.faults, m = self.faults + 1, i
                        break
                got = [self.rows(seq, n + int(path[i]), n + int(path[i]) + 1) for i in range(m)]
                for i, (k, v) in enumerate(got):
                    self.put(seq, n + i, k, v)
            self.len[seq] = n + m
            self.next[seq] += m if advance < 0 else advance

    def own(self, seq, rows):
        """Rows len .. len + rows - 1 all lie in pages that the sequence holds alone."""
        n, end = int(self.len[seq]) // self.page, -(-(int(self.len[seq]) + rows) // self.page)
        return end <= self.held[seq] and all(0 <= p < len(self.refs) and self.refs[p] == 1 for p in self.table[seq, n:end])

    def rows(self, seq, a, b):
        """K and V [Hkv][b - a][d] of rows a .. b-1."""
        at = [(int(self.table[seq, t // self.page]), t % self.page) for t in range(a, b)]
        return tuple(np.stack([x[p, :, i] for p, i in at], 1) if at else x[0, :, :0] for x in (self.k, self.v))

    def put(self, seq, a, k, v):
        for t in range(k.shape[1]):
            p, i = int(self.table[seq, (a + t) // self.page]), (a + t) % self.page
            assert self.refs[p] == 1
            self.k[p, :, i], self.v[p, :, i] = k[:, t], v[:, t]

    def check(self):
        """Pages are counted right, and every page is either on the stack or held."""
        count = np.zeros_like(self.refs)
        for seq in range(len(self.held)):
            assert self.held[seq] * self.page >= self.len[seq]
            mine = self.table[seq, : self.held[seq]]
            assert len(set(mine.tolist())) == len(mine)
            count[mine] += 1
        assert np.array_equal(count, self.refs)
        assert sorted(self.free[: self.n_free].tolist()) == np.flatnonzero(count == 0).tolist()


def axes(sections, dealt):
    """Axis of each pair."""
    out, left, turn = [], list(sections), 0
    while sum(left):
        if dealt:
            if left[turn]:
                out.append(turn)
                left[turn] -= 1
            turn = (turn + 1) % len(left)
        else:
            a = next(i for i, n in enumerate(left) if n)
            out.append(a)
            left[a] -= 1
    return out


def rope_axes(x, pos, freqs, axis, interleaved, amp=1.0):
    """x [rows][heads][d], pos [axes][rows], axis of each pair: the rotated rows in float64."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = len(freqs)
    for j, th in enumerate(freqs):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        at = np.asarray(pos[axis[j]], np.float64) * th
        c, s = amp * np.cos(at)[:, None], amp * np.sin(at)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def ancestors(parent):
    """[N][N] truth values: node i sees node j; and the depths."""
    N = len(parent)
    see = np.zeros((N, N), bool)
    for i in range(N):
        j = i
        while True:
            see[i, j] = True
            if not 0 <= parent[j] < j:
                break
            j = parent[j]
    return see, see.sum(1) - 1


def pack(see, words):
    """Rows of truth values as int32 words, bit j % 32 of word j / 32."""
    out = np.zeros((see.shape[0], words), np.uint32)
    for i, j in zip(*np.nonzero(see)):
        out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def tree_attn(q, k, v, see):
    """q [N][Hq][d]; k, v [Hkv][ctx + N][d]; see [N][N]: token i sees the context and tokens j with see[i][j].
    Zeros for a row that sees nothing."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    N, Hq, d = q.shape
    G, ctx = Hq // k.shape[0], k.shape[1] - N
    o = np.zeros((N, Hq, d))
    for i in range(N):
        keys = np.concatenate([np.arange(ctx), ctx + np.flatnonzero(see[i])])
        if len(keys) == 0:
            continue
        for h in range(Hq):
            s = k[h // G, keys] @ q[i, h] / np.sqrt(d)
            e = np.exp(s - s.max())
            o[i, h] = (e / e.sum()) @ v[h // G, keys]
    return o


def accept_tree(logits, token, parent, n):
    """(path, tokens) of the longest path from node 0 whose tokens the predictions agree with."""
    path, out = [], []
    cur = 0 if n > 0 else None
    while cur is not None:
        row = np.where(np.isnan(logits[cur]), -np.inf, logits[cur])
        pick = 0 if np.isnan(logits[cur]).all() else int(np.flatnonzero((row == row.max()) & ~np.isnan(logits[cur]))[0])
        path.append(cur)
        out.append(pick)
        cur = next((j for j in range(cur + 1, n) if parent[j] == cur and token[j] == pick), None)
    return path, out
