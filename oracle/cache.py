"""ORACLE -- test infrastructure only.

The paged cache of the verification pass, written out plainly with Python lists and
64-bit arithmetic.  A state is three lists: `table` (each row its page ids, -1 for none),
`len` (tokens kept, negative for a vacant row) and `ref` (rows that hold each page).  Page
contents are arrays [layers, n_pages, heads, page, dim] in token order; pack_k / pack_v
give the block order in which the library keeps them.

Readings:
  * pages are handed out lowest first, to the requests in order; a request is served if
    the pages that it and all requests before it need exist;
  * a token that a row does not see has no influence, whatever its values;
  * page ids outside the cache are tokens that are not there.
"""
from __future__ import annotations

import math

import numpy as np

BAD_PAGE, BAD_ROW, NO_PAGES = 32, 64, 128


def pack_k(x):
    """[..., page, D] -> [..., page/16, D/8, 16, 8]"""
    *lead, page, D = x.shape
    y = x.reshape(*lead, page // 16, 16, D // 8, 8)
    return np.ascontiguousarray(np.swapaxes(y, -3, -2))


def pack_v(x):
    """[..., page, D] -> [..., page/16, D, 16]"""
    *lead, page, D = x.shape
    return np.ascontiguousarray(np.swapaxes(x.reshape(*lead, page // 16, 16, D), -2, -1))


def unpack_k(y):
    *lead, blocks, chunks, _, _ = y.shape
    return np.ascontiguousarray(np.swapaxes(y, -3, -2)).reshape(*lead, blocks * 16, chunks * 8)


def unpack_v(y):
    *lead, blocks, D, _ = y.shape
    return np.ascontiguousarray(np.swapaxes(y, -2, -1)).reshape(*lead, blocks * 16, D)


def _pages(tokens, page):
    return -(-tokens // page)


def _held(row):
    n = 0
    while n < len(row) and row[n] >= 0:
        n += 1
    return n


def reserve(table, length, ref, offsets, lead, page):
    """Changes table and ref; returns (granted, status)."""
    free = [p for p, n in enumerate(ref) if n <= 0]
    told, status, granted = 0, 0, []
    for r in range(len(offsets) - 1):
        row, ln, n = table[r], length[r], offsets[r + 1] - offsets[r] + lead
        if ln < 0:
            granted.append(0)
            continue
        if n < 0 or _pages(ln, page) > _held(row):
            status |= BAD_ROW
            granted.append(0)
            continue
        held = _held(row)
        want = _pages(ln + n, page)
        if want > len(row):
            status |= NO_PAGES
            granted.append(0)
            continue
        need = max(0, want - held)
        ok = need == 0 or told + need <= len(free)
        if ok:
            for i in range(need):
                row[held + i] = free[told + i]
                ref[free[told + i]] = 1
        else:
            status |= NO_PAGES
        told += need
        granted.append(int(ok))
    return granted, status


def _drop(table, ref, r, first):
    status = 0
    for i in range(first, len(table[r])):
        p, table[r][i] = table[r][i], -1
        if p < 0:
            continue
        if p >= len(ref) or ref[p] <= 0:
            status |= BAD_PAGE
        else:
            ref[p] -= 1
    return status


def trim(table, length, ref, rows, keep, page):
    status = 0
    for r, k in zip(rows, keep):
        if not 0 <= r < len(table):
            status |= BAD_ROW
            continue
        status |= _drop(table, ref, r, _pages(max(k, 0), page))
        length[r] = min(length[r], k if k >= 0 else -1)
    return status


def commit(table, length, ref, accept, lead, page, granted=None):
    status = 0
    for r, a in enumerate(accept):
        if length[r] < 0 or (granted is not None and not granted[r]):
            continue
        kept = length[r] + lead + a
        first = _pages(kept, page)
        if a < 0 or first > len(table[r]) or (first > 0 and table[r][first - 1] < 0):
            status |= BAD_ROW
            continue
        status |= _drop(table, ref, r, first)
        length[r] = kept
    return status


def fork(table, length, ref, src, dst, deep, page):
    """Returns (forked, status, [(page copied from, page copied to)])."""
    free = [p for p, n in enumerate(ref) if n <= 0]
    old, old_len = [list(t) for t in table], list(length)
    told, status, forked, pairs = 0, 0, [], []
    for i, (a, d) in enumerate(zip(src, dst)):
        good = 0 <= a < len(table) and 0 <= d < len(table) and a != d and d not in dst[:i]
        good = good and old_len[a] >= 0 and old_len[d] <= 0 and old[d][0] < 0
        total = _pages(old_len[a], page) if good else 0
        if not good or total > _held(old[a]):
            status |= BAD_ROW
            forked.append(0)
            continue
        whole = 0 if deep else old_len[a] // page
        need = total - whole
        ok = told + need <= len(free)
        if ok:
            for j in range(whole):
                table[d][j] = old[a][j]
                ref[old[a][j]] += 1
            for j in range(need):
                p = free[told + j]
                table[d][whole + j] = p
                ref[p] = 1
                pairs.append((old[a][whole + j], p))
            length[d] = old_len[a]
        else:
            status |= NO_PAGES
        told += need
        forked.append(int(ok))
    return forked, status, pairs


def compact(table, ref):
    """Returns (page_map, n_live, status, [(from, to)])."""
    n = len(ref)
    live = [p for p in range(n) if ref[p] > 0]
    holes = [p for p in range(len(live)) if ref[p] <= 0]
    moves = list(zip([p for p in live if p >= len(live)], holes))
    page_map = [p if ref[p] > 0 else -1 for p in range(n)]
    for a, b in moves:
        page_map[a] = b
        ref[b], ref[a] = ref[a], 0
    status = 0
    for row in table:
        for i, p in enumerate(row):
            if p < 0:
                continue
            row[i] = page_map[p] if p < n else -1
            if row[i] < 0:
                status |= BAD_PAGE
    return page_map, len(live), status, moves


def rows_of(offsets, lead, r):
    return offsets[r] + lead * r, offsets[r + 1] + lead * (r + 1)


def append(k, v, table, length, k_new, v_new, offsets, lead):
    """k, v [n_pages, heads, page, D] of one layer, changed in place."""
    page = k.shape[2]
    for r in range(len(offsets) - 1):
        a, b = rows_of(offsets, lead, r)
        if length[r] < 0:
            continue
        for j in range(b - a):
            p = length[r] + j
            k[table[r][p // page], :, p % page] = k_new[a + j]
            v[table[r][p // page], :, p % page] = v_new[a + j]


def attend(q, k, v, table, length, offsets, lead, scale):
    """q [rows, H, D], k, v [n_pages, heads, page, D] in float64.  Returns out [rows, H, D],
    lse [rows, H], and for error bounds spread [rows, H, D] = softmax-weighted |V| and
    reach [rows, H] = the largest scale * sum |q||K|, -1 for rows of no request; rows that
    see nothing are 0 with lse -inf."""
    rows, H, D = q.shape
    n_pages, heads, page, _ = k.shape
    G = H // heads
    out, spread = np.full((rows, H, D), np.nan), np.full((rows, H, D), np.nan)
    lse, reach = np.full((rows, H), np.nan), np.full((rows, H), -1.0)
    for r in range(len(offsets) - 1):
        a, b = rows_of(offsets, lead, r)
        for t in range(a, b):
            last = length[r] + (t - a) if length[r] >= 0 else -1
            seen = [(table[r][p // page], p % page) for p in range(last + 1)]
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
