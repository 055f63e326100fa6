"""Pins of the trees' oracle: worked trees, closed forms of rotary positions and of the
target's choice."""
import math

import numpy as np

from oracle import cache as oc
from oracle import tree as ot


def test_worked_merge_plan_accept():
    # chains 5 6 7, 5 6 8 and 9 1 (cut to 1): 5-6-7, a second child 8 of 6, and 9 beside 5
    got = ot.merge([[[5, 6, 7], [5, 6, 8], [9, 1, 1]], [[4, 4, 4], [4, 4, 4], [4, 5, 6]]], [[3, 3, 1], [2, 3, 0]])
    assert got == ([5 - 0, 3], [0, 5, 8], [5, 6, 7, 8, 9, 4, 4, 4], [-1, 0, 1, 2, 2, 0, -1, 0, 1, 2], 0)
    counts, offsets, drafts, parent, _ = got
    depth, anc = [0] * 10, [0] * 10
    assert ot.plan(parent, offsets, 1, 64, depth, anc) == 0
    assert depth == [0, 1, 2, 3, 3, 1, 0, 1, 2, 3]
    assert anc == [1, 3, 7, 15, 23, 33, 1, 3, 7, 15]
    # the target says 5 6 8 and then 2; in the second request something else at once
    target = [5, 6, 8, 0, 2, 0, 3, 4, 4, 4]
    a, path, nxt, out, st = ot.accept(drafts, offsets, parent, target, 3)
    assert (a, path, nxt, out, st) == ([3, 0], [[1, 2, 4], [-1] * 3], [2, 3], [[5, 6, 8, 2], [3, -1, -1, -1]], 0)
    a, path, nxt, out, st = ot.accept(drafts, offsets, parent, target, 2)  # no more than two
    assert a[0] == 2 and path[0] == [1, 2] and nxt[0] == 8 and out[0] == [5, 6, 8]
    assert ot.merge([[[1, 2]]], [[3]])[4] == ot.BAD_ROW


def test_plan_of_what_is_no_tree():
    depth, anc = [7] * 6, [7] * 6
    # node 2 names itself, 3 hangs on it; 4 is a second root
    assert ot.plan([-1, 0, 2, 2, -1, 4], [0, 5], 1, 64, depth, anc) == ot.BAD_ROW
    assert depth == [0, 1, 0, 0, 0, 1] and anc == [1, 3, 0, 0, 16, 48]


def test_keep_path_moves_nodes_together():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 3, 1, 16, 4)), rng.standard_normal((2, 3, 1, 16, 4))
    old = k.copy()
    table, ref = [[2, 0, -1]], [1, 0, 1]
    # 14 tokens kept: node 0 at 14, 1 at 15, the others in page 0
    assert ot.keep_path(k, v, table, [14], ref, [[1, 4, 7, -1]], [3], 1) == 0
    np.testing.assert_array_equal(k[:, 2], old[:, 2])
    np.testing.assert_array_equal(k[:, 0, :, 0], old[:, 0, :, 2])
    np.testing.assert_array_equal(k[:, 0, :, 1], old[:, 0, :, 5])
    np.testing.assert_array_equal(k[:, 0, :, 2:], old[:, 0, :, 2:])
    assert ot.keep_path(k, v, table, [14], ref, [[2, 2]], [2], 1) == ot.BAD_ROW
    assert ot.keep_path(k, v, table, [40], ref, [[2, 9]], [2], 1) == ot.BAD_ROW  # past the table
    assert ot.keep_path(k, v, table, [20], ref, [[12]], [1], 1) == ot.BAD_PAGE   # in a page that is not there


def test_a_chain_attends_as_the_cache_does():
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((6, 4, 8))
    table, length, offsets = [[1, 3], [2, 0]], [18, 5], [0, 2, 4]
    chain = [(2 << j) - 1 for j in (0, 1, 2, 0, 1, 2)]
    for x, y in zip(oc.attend(q, k, v, table, length, offsets, 1, 0.3), ot.attend(q, k, v, table, length, offsets, 1, 0.3, chain)):
        np.testing.assert_array_equal(x, y)
    out, lse, _, _ = ot.attend(q, k, v, table, length, offsets, 1, 0.3, [0] * 6)
    assert not out.any() and (lse == -math.inf).all()


def test_rotary_closed_forms():
    np.testing.assert_allclose(ot.frequencies(8), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    np.testing.assert_allclose(ot.frequencies(8, scaling="linear", factor=4.0), [0.25, 0.025, 0.0025, 0.00025], rtol=1e-14)
    # far inside the original length a pair keeps its frequency, far outside it is divided
    for how in ("bands", "ramp"):
        f = ot.frequencies(64, 10000.0, how, 8.0, 4096, 1.0, 32.0) / ot.frequencies(64)
        assert f[0] == 1.0 and abs(f[-1] - 0.125) < 1e-15 and (np.diff(f) <= 1e-15).all()
    x = np.zeros((1, 1, 16))
    x[0, 0, 0], x[0, 0, 9] = 1.0, 2.0
    y, _ = ot.rotate(x, [3], ot.frequencies(16), 16, 0, False, 1.0)  # dims 0, 8 and 1, 9 pair
    np.testing.assert_allclose([y[0, 0, 0], y[0, 0, 8]], [math.cos(3.0), math.sin(3.0)], rtol=1e-14)
    w = 3.0 * 10.0 ** -0.5
    np.testing.assert_allclose([y[0, 0, 1], y[0, 0, 9]], [-2 * math.sin(w), 2 * math.cos(w)], rtol=1e-13)
    # products of turned vectors depend on the distance alone
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    for inter in (False, True):
        dots = [(ot.rotate(q, [a], ot.frequencies(16), 16, 0, inter, 1.0)[0] * ot.rotate(k, [b], ot.frequencies(16), 16, 0, inter, 1.0)[0]).sum()
                for a, b in ((5, 2), (1003, 1000))]
        np.testing.assert_allclose(dots[0], dots[1], rtol=1e-11)


def test_worked_choices():
    x = np.array([3.0, 4.0, -1.0, 4.0, 0.0])
    assert ot.choose(x, [])[0] == 1                                     # the lowest of equal ones
    assert ot.choose(x, [], prompt={1}, repetition=2.0)[0] == 3
    t, y = ot.choose(x, [1, 1], prompt={2}, count={3: 2}, repetition=2.0, presence=0.5, frequency=0.25)
    assert t == 0 and y.tolist() == [3.0, 2.0 - 0.5 - 0.5, -2.0, 2.0 - 0.5 - 0.5, 0.0]
    assert ot.choose(x, [], bias={4: 5.0})[0] == 4
    t, y = ot.choose(x, [], allowed=np.array([0, 0, 1, 0, 1], bool))
    assert t == 4 and y.tolist() == [-np.inf, -np.inf, -1.0, -np.inf, 0.0]
    assert ot.choose(x, [], allowed=np.zeros(5, bool))[0] == 0
    assert ot.choose(np.array([1.0, np.nan, np.nan]), [])[0] == 1
    assert ot.choose(np.array([1.0, np.nan]), [], allowed=np.array([1, 0], bool))[0] == 0
    assert ot.choose(np.array([-np.inf, -np.inf]), [], allowed=np.array([0, 1], bool))[0] == 1


def test_history_arrays():
    h = ot.History(2, 40)
    assert h.add([[1, 1, -1, 39]], True, [1]) == 0 and h.add([[2, 40]], False, [1]) == ot.BAD_ROW
    seen, count = h.arrays()
    assert seen.shape == (2, 2, 4) and count[1, 1] == 2 and count[1, 39] == 1 and count.sum() == 3
    assert seen[1, 1].tolist() == [2, 1 << 7, 0, 0] and seen[1, 0].tolist() == [4, 0, 0, 0] and not seen[0].any()
    assert h.clear([1, 2]) == ot.BAD_ROW and not h.arrays()[0].any()
