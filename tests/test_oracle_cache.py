"""Pins of the paged cache's oracle: the packed order round-trips, the bookkeeping keeps
its counts equal to the tables, worked cases, and attention's closed forms."""
import copy

import numpy as np
import pytest

from oracle import cache as oc


def _counts(table, n_pages):
    ref = [0] * n_pages
    for row in table:
        for p in row:
            if p >= 0:
                ref[p] += 1
    return ref


def test_packed_order():
    x = np.arange(2 * 3 * 32 * 64).reshape(2, 3, 32, 64)
    k, v = oc.pack_k(x), oc.pack_v(x)
    assert k.shape == (2, 3, 2, 8, 16, 8) and v.shape == (2, 3, 2, 64, 16)
    assert k[1, 2, 1, 5, 7, 3] == x[1, 2, 16 + 7, 5 * 8 + 3]
    assert v[1, 2, 1, 43, 7] == x[1, 2, 16 + 7, 43]
    np.testing.assert_array_equal(oc.unpack_k(k), x)
    np.testing.assert_array_equal(oc.unpack_v(v), x)


def test_worked_reserve_commit():
    # pages of 16: request 0 keeps 15 tokens in page 3 and needs one more page for 1 + 2 rows;
    # request 1 has room; request 2 is vacant; request 3 needs two pages, of which one is left
    table = [[3, -1, -1], [0, -1, -1], [-1] * 3, [-1] * 3]
    length, ref = [15, 2, -1, 0], [1, 0, 0, 1]
    granted, st = oc.reserve(table, length, ref, [0, 2, 4, 6, 40], 1, 16)
    assert granted == [1, 1, 0, 0] and st == oc.NO_PAGES
    assert table[0] == [3, 1, -1] and ref == [1, 1, 0, 1] and table[3] == [-1] * 3
    assert oc.commit(table, length, ref, [0, 1, 5, -1], 1, 16) == oc.BAD_ROW
    assert length == [16, 4, -1, 0] and table[0] == [3, -1, -1] and ref == [1, 0, 0, 1]


def test_worked_fork_and_compact():
    table = [[5, 2, 7, -1], [-1] * 4, [-1] * 4, [-1] * 4]
    length, ref = [40, 0, -1, 0], [0, 0, 1, 0, 0, 1, 0, 1]
    forked, st, pairs = oc.fork(table, length, ref, [0, 0, 0, 9], [1, 2, 1, 3], False, 16)
    assert forked == [1, 1, 0, 0] and st == oc.BAD_ROW
    assert table[1] == [5, 2, 0, -1] and table[2] == [5, 2, 1, -1] and length == [40, 40, 40, 0]
    assert pairs == [(7, 0), (7, 1)] and ref == _counts(table, 8)
    page_map, n_live, st, moves = oc.compact(table, ref)
    assert n_live == 5 and st == 0 and moves == [(5, 3), (7, 4)]
    assert table[0] == [3, 2, 4, -1] and ref == _counts(table, 8)
    assert page_map == [0, 1, 2, -1, -1, 3, -1, 4]


@pytest.mark.parametrize("seed", range(6))
def test_counts_follow_the_tables(seed):
    rng = np.random.default_rng(seed)
    R, width, page, n_pages = 9, 7, 16, 40
    table, length, ref = [[-1] * width for _ in range(R)], [0] * R, [0] * n_pages
    for _ in range(12):
        offsets = np.concatenate([[0], np.cumsum(rng.integers(0, 20, R))]).tolist()
        granted, _ = oc.reserve(table, length, ref, offsets, 1, page)
        accept = [int(rng.integers(0, offsets[r + 1] - offsets[r] + 1)) if granted[r] else -1 for r in range(R)]
        before = copy.deepcopy(table)
        oc.commit(table, length, ref, accept, 1, page)
        assert all(row[:3] == old[:3] for row, old, ln in zip(table, before, length) if ln > 48)
        oc.trim(table, length, ref, [int(rng.integers(0, R))], [int(rng.integers(-1, 30))], page)
        src, dst = rng.permutation(R)[:2].tolist()
        oc.fork(table, length, ref, [src], [dst], bool(rng.integers(2)), page)
        if rng.random() < 0.4:
            oc.compact(table, ref)
        assert ref == _counts(table, n_pages)
        assert all(oc._held(row) * page >= ln for row, ln in zip(table, length))


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((4, 2, 16, 8))
    table, length, offsets = [[2, 0], [1, -1], [3, 3]], [17, -1, 0], [0, 2, 3, 3]
    q = np.zeros((6, 4, 8))
    out, lse, _, _ = oc.attend(q, k, v, table, length, offsets, 1, 0.3)
    tokens = np.concatenate([v[2], v[0]], axis=1)  # equal scores give the mean of V
    np.testing.assert_allclose(out[1, 3], tokens[1, :19].mean(0))
    np.testing.assert_allclose(lse[1, 3], np.log(19))
    assert (out[3:5] == 0).all() and np.isneginf(lse[3:5]).all()       # a vacant request's rows
    np.testing.assert_allclose(out[5], np.repeat(v[3][:, 0], 2, axis=0))  # one token: its V
    q[0, 1] = 1000 * k[2, 0, 5]  # one token outweighs the rest
    out, lse, _, _ = oc.attend(q, k, v, table, length, offsets, 1, 1.0)
    best = int(np.argmax(np.concatenate([k[2], k[0]], axis=1)[0, :18] @ k[2, 0, 5]))
    np.testing.assert_allclose(out[0, 1], tokens[0, best], atol=1e-12)
