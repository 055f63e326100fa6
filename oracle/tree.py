"""ORACLE -- test infrastructure only.

Trees of drafts, rotary positions and the target's choice, written out plainly: Python lists
and sets for what is counted, 64-bit (angles: 80-bit) arithmetic for what is computed.  The
paged cache's states are those of oracle.cache.

Readings:
  * a tree's nodes are numbered by chain, then by position, each beginning once;
  * a node whose parent is not an earlier one (or -1) sees nothing, nor does what hangs on it;
  * penalties come in the order repetition, frequency, presence, bias, mask, each a rounded
    64-bit operation; drafts on a row's path count like answered tokens.
"""
from __future__ import annotations

import math

import numpy as np

from .cache import BAD_PAGE, BAD_ROW, rows_of

BAD_ALLOCATION, NO_TOKEN = 16, 256
NODES = 64


def merge(chains, lens):
    """chains [R][S] lists of K tokens, lens [R][S].  Returns (counts, offsets, drafts, parents, status)."""
    counts, offsets, drafts, parents, status = [], [0], [], [], 0
    for chain, ln in zip(chains, lens):
        names = {(): 0}
        parents.append(-1)
        n = 0
        for tokens, upto in zip(chain, ln):
            if not 0 <= upto <= len(tokens):
                status, upto = status | BAD_ROW, 0
            for i in range(upto):
                name = tuple(tokens[:i + 1])
                if name not in names:
                    n += 1
                    names[name] = n
                    drafts.append(tokens[i])
                    parents.append(names[name[:-1]])
        counts.append(n)
        offsets.append(offsets[-1] + n)
    return counts, offsets, drafts, parents, status


def plan(parent, offsets, lead, max_new, depth, anc):
    """Depths and words (Python integers) into the lists depth and anc; returns status."""
    status = 0
    for r in range(len(offsets) - 1):
        a, b = rows_of(offsets, lead, r)
        if offsets[r] < 0 or not 0 <= b - a <= max_new or b > len(parent):
            status |= BAD_ROW
            continue
        for j in range(b - a):
            p = parent[a + j]
            if p < -1 or p >= j or (p >= 0 and anc[a + p] == 0):
                depth[a + j] = anc[a + j] = 0
                status |= BAD_ROW
            else:
                depth[a + j] = 0 if p < 0 else depth[a + p] + 1
                anc[a + j] = (0 if p < 0 else anc[a + p]) | 1 << j
    return status


def accept(drafts, offsets, parent, target, K):
    """Returns (accept_len, path, next_prev0, out_tokens, status)."""
    got, status = ([], [], [], []), 0
    for r in range(len(offsets) - 1):
        o, L = offsets[r], offsets[r + 1] - offsets[r]
        way, bonus, said = [], -1, []
        if o < 0 or not 0 <= L < NODES or o + L > len(drafts):
            status |= BAD_ALLOCATION
        else:
            at = 0
            while True:
                bonus = target[o + r + at]
                nexts = [j for j in range(at + 1, L + 1) if parent[o + r + j] == at and drafts[o + j - 1] == bonus]
                if len(way) == K or not nexts:
                    break
                at = nexts[0]
                way.append(at)
                said.append(bonus)
            said.append(bonus)
        for x, y in zip(got, (len(way), way + [-1] * (K - len(way)), bonus, said + [-1] * (K + 1 - len(said)))):
            x.append(y)
    return (*got, status)


def keep_path(k, v, table, length, ref, path, accept_len, lead, granted=None):
    """k, v [layers, n_pages, heads, page, D], changed in place; returns status."""
    page, status = k.shape[3], 0
    for r, n in enumerate(accept_len):
        if length[r] < 0 or (granted and not granted[r]):
            continue
        K, row = len(path[r]), table[r]
        way = path[r][:n] if 0 <= n <= K else None
        if way is None or any(b <= a for a, b in zip([lead - 1] + way, way)) or \
                any(j >= NODES or (length[r] + j) // page >= len(row) for j in way):
            status |= BAD_ROW
            continue
        moves = [(length[r] + j, length[r] + lead + i) for i, j in enumerate(way) if j != lead + i]
        pages = [(row[a // page], row[b // page]) for a, b in moves]
        if any(not 0 <= p < k.shape[1] for pair in pages for p in pair) or any(ref[q] > 1 for _, q in pages):
            status |= BAD_PAGE
            continue
        old_k, old_v = k.copy(), v.copy()
        for (a, b), (p, q) in zip(moves, pages):
            k[:, q, :, b % page], v[:, q, :, b % page] = old_k[:, p, :, a % page], old_v[:, p, :, a % page]
    return status


def attend(q, k, v, table, length, offsets, lead, scale, anc):
    """oracle.cache.attend for trees: anc [rows] Python integers."""
    rows, H, D = q.shape
    n_pages, heads, page, _ = k.shape
    G = H // heads
    out, spread = np.full((rows, H, D), np.nan), np.full((rows, H, D), np.nan)
    lse, reach = np.full((rows, H), np.nan), np.full((rows, H), -1.0)
    for r in range(len(offsets) - 1):
        a, b = rows_of(offsets, lead, r)
        for t in range(a, b):
            at = []
            if length[r] >= 0 and anc[t]:
                at = list(range(length[r])) + [length[r] + i for i in range(b - a) if anc[t] >> i & 1]
            seen = [(table[r][p // page], p % page) for p in at]
            seen = [(i, s) for i, s in seen if 0 <= i < n_pages]
            if not seen:
                out[t], spread[t], lse[t], reach[t] = 0.0, 0.0, -math.inf, 0.0
                continue
            ids, slots = np.array(seen).T
            for h in range(H):
                K, V = k[ids, h // G, slots], v[ids, h // G, slots]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (K @ q[t, h])
                    m = s.max()
                    w = np.exp(s - m)
                    out[t, h] = (w[:, None] * V).sum(0) / w.sum()
                    spread[t, h] = (w[:, None] * np.abs(V)).sum(0) / w.sum()
                lse[t, h] = m + math.log(w.sum()) if np.isfinite(m) else m
                reach[t, h] = scale * (np.abs(K) @ np.abs(q[t, h])).max()
    return out, lse, spread, reach


def frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=0.0, low=0.0, high=0.0):
    """Radians a token of each pair, pair by pair."""
    got = []
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        wave = 2.0 * math.pi / f  # tokens a turn
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            turns = original / wave
            if turns <= low:
                f = f / factor
            elif turns < high:
                s = (turns - low) / (high - low)
                f = (1.0 - s) * f / factor + s * f
        elif scaling == "ramp":
            def pair(x):
                return dim * math.log(original / (x * 2.0 * math.pi)) / (2.0 * math.log(base))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), dim - 1)
            s = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f / factor * s + f * (1.0 - s)
        got.append(f)
    return np.array(got)


def rotate(x, pos, freq, dim, first, interleaved, attention):
    """x [n, heads, D] in float64, pos [n] integers; returns (turned, |a| + |b| of each dim's pair)."""
    y, reach = x.copy(), np.abs(x)
    half = dim // 2
    a, b = (first + 2 * np.arange(half), first + 2 * np.arange(half) + 1) if interleaved else \
        (first + np.arange(half), first + half + np.arange(half))
    t = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble)
    c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
    y[:, :, a] = attention * (x[:, :, a] * c - x[:, :, b] * s)
    y[:, :, b] = attention * (x[:, :, a] * s + x[:, :, b] * c)
    reach[:, :, a] = reach[:, :, b] = abs(attention) * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
    return y, reach


class History:
    """Sets and counts of each row."""

    def __init__(self, rows, V):
        self.prompt, self.count, self.V = [set() for _ in range(rows)], [{} for _ in range(rows)], V

    def clear(self, rows):
        status = 0
        for r in rows:
            if not 0 <= r < len(self.prompt):
                status |= BAD_ROW
                continue
            self.prompt[r], self.count[r] = set(), {}
        return status

    def add(self, tokens, answered, rows):
        status = 0
        for r, row in zip(rows, tokens):
            if not 0 <= r < len(self.prompt):
                status |= BAD_ROW
                continue
            for v in row:
                if v >= self.V:
                    status |= BAD_ROW
                elif v >= 0 and answered:
                    self.count[r][v] = self.count[r].get(v, 0) + 1
                elif v >= 0:
                    self.prompt[r].add(v)
        return status

    def arrays(self):
        rows, words = len(self.prompt), (self.V + 127) // 128 * 4
        seen, count = np.zeros((rows, 2, words * 32), bool), np.zeros((rows, self.V), np.int32)
        for r in range(rows):
            seen[r, 0, list(self.prompt[r])] = True
            seen[r, 1, list(self.count[r])] = True
            for v, n in self.count[r].items():
                count[r, v] = n
        return np.packbits(seen, axis=2, bitorder="little").view(np.int32), count


def choose(logits, path, prompt=(), count=None, repetition=1.0, presence=0.0, frequency=0.0, bias=None, allowed=None):
    """One row: logits [V] float64, path the drafts that it has behind it, prompt a set, count and bias dicts,
    allowed [V] truth values or None.  Returns (token, processed logits); token 0 where nothing is
    allowed, the lowest of values that are all -inf."""
    x = logits.copy()
    times = dict(count or {})
    for v in path:
        if 0 <= v < len(x):
            times[v] = times.get(v, 0) + 1
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        for v in set(prompt) | set(times):
            n = times.get(v, 0)
            x[v] = x[v] / repetition if x[v] > 0 else x[v] * repetition
            if n > 0:
                x[v] = x[v] - np.float64(frequency) * n
                x[v] = x[v] - presence
        for v, b in (bias or {}).items():
            x[v] = x[v] + b
    free = np.arange(len(x)) if allowed is None else np.nonzero(allowed)[0]
    y = np.full_like(x, -np.inf)
    y[free] = x[free]
    if not len(free):
        return 0, y
    nan = free[np.isnan(x[free])]
    best = nan[0] if len(nan) else free[np.argmax(x[free])]
    return int(best), y
