"""Plain CPU oracle of the caches that grow, are shared and shrink while requests decode: rotary
positions, attention over a shared prefix, attention weights gathered per cached row, eviction.

Test infrastructure only, like the rest of this package. Everything is float64 and written from the
definitions in include/vc.h; selection is a sort.
"""
from __future__ import annotations

import numpy as np


def rope_freqs(kind, rot, base, factor=1.0, orig_ctx=0, low=1.0, high=4.0):
    """Radians a position of the rot / 2 pairs."""
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for j in range(rot // 2):
        th = base ** (-2.0 * j / rot)
        if kind == "linear":
            th /= factor
        if kind == "bands":
            turns = orig_ctx * th / (2 * np.pi)
            if turns < low:
                th = th / factor
            elif turns <= high:
                m = (turns - low) / (high - low)
                th = m * th + (1 - m) * th / factor
        out.append(th)
    return np.array(out)


def rope(x, pos, freqs, interleaved, amp=1.0):
    """x [rows][heads][d], pos [rows]: the rotated rows in float64."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = len(freqs)
    for j, th in enumerate(freqs):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c = amp * np.cos(np.asarray(pos, np.float64) * th)[:, None]
        s = amp * np.sin(np.asarray(pos, np.float64) * th)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def live_attn(q, k, v, prefix=None):
    """q [rows][Hq][d]; k, v [Hkv][n][d]; prefix (pk, pv) [Hkv][P][d] or None. Row i sees the prefix
    and own rows t <= n - rows + i. Returns (o [rows][Hq][d], w [Hkv][n]): the outputs, zeros for a
    row that sees nothing, and the weight every own row got."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    rows, Hq, d = q.shape
    Hkv, n = k.shape[0], k.shape[1]
    G = Hq // Hkv
    o, w = np.zeros((rows, Hq, d)), np.zeros((Hkv, n))
    for i in range(rows):
        seen = max(0, n - rows + i + 1)
        for h in range(Hq):
            kk, vv = k[h // G, :seen], v[h // G, :seen]
            P = 0
            if prefix is not None:
                P = prefix[0].shape[1]
                kk = np.concatenate([np.asarray(prefix[0][h // G], np.float64), kk])
                vv = np.concatenate([np.asarray(prefix[1][h // G], np.float64), vv])
            if len(kk) == 0:
                continue
            s = kk @ q[i, h] / np.sqrt(d)
            e = np.exp(s - s.max())
            p = e / e.sum()
            o[i, h] = p @ vv
            w[h // G, :seen] += p[P:]
    return o, w


def evict(score, pos, keep, sink, recent_from):
    """One head's n rows: (holes, moves) ascending, so that row moves[j] goes to row holes[j]."""
    n = len(score)
    if n <= keep:
        return [], []

    def rank(i):  # smaller is better
        if pos[i] < sink or pos[i] >= recent_from:
            return (0, 0.0, i)
        if np.isnan(score[i]):
            return (2, 0.0, i)
        return (1, -float(score[i]), i)

    kept = set(sorted(range(n), key=rank)[:keep])
    return [i for i in range(keep) if i not in kept], [i for i in range(keep, n) if i in kept]
