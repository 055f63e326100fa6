"""Attention over the paged cache where scores are not finite: a NaN in a query or in a key
that a row sees makes that row's result with the key's heads NaN, whichever form computes it,
however its keys are split over waves and workgroups, and behind a shared prefix.  The
oracle (64 bits) gives NaN there by itself; all other rows and heads keep their bounds."""
import math

import numpy as np
import pytest

import cache_util as cu
from test_gpu_attend import Case

pytestmark = pytest.mark.gpu

# Few columns (waves stream keys), and more than 64 (keys through LDS for all waves); contexts
# of one workgroup and of many; whole pages of the first ones shared.
SHAPES = {
    "one wave": dict(lens=[5, 20], rows=[1, 2]),
    "few rows": dict(lens=[32, 100, 128], rows=[1, 3, 1]),
    "few rows, split": dict(lens=[3000, 1500], rows=[2, 1]),
    "few rows, prefix": dict(lens=[144, 150, 144, 260], rows=[1, 2, 1, 3], groups=[(3, 9)]),
    "two tiles, split": dict(lens=[2100, 70], rows=[16, 20]),
    "many rows": dict(lens=[0, 64, 10], rows=[90, 70, 40]),
    "many rows, split": dict(lens=[2000, 256], rows=[75, 40]),
    "many rows, prefix": dict(lens=[9 * 16, 9 * 16 + 64, 700], rows=[40, 70, 36], groups=[(2, 9)]),
}


def _case(seed, shape, D, dtype):
    s = SHAPES[shape]
    return Case(seed, s["lens"], s["rows"], 4, 2, D, dtype, 16, groups=s.get("groups", ()))


def _check(c, want, seen):
    """`seen`: (row, head) of NaN results."""
    assert seen and all(np.isnan(want[0][t, h]).all() and np.isnan(want[1][t, h]) for t, h in seen)
    assert np.isfinite(want[0]).any()
    c.check(want=want)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_a_query_that_is_not_a_number(shape, dtype, D):
    print("attend, NaN in q", shape, dtype, D, flush=True)
    c = _case(31, shape, D, dtype)
    seen = [(0, 1), (c.rows - 1, 2)]
    for t, h in seen:
        c.q[t, h, D // 2 + h] = math.nan
    _check(c, c.want(), seen)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_the_last_key_of_a_row_is_not_a_number(shape, dtype, D):
    # the key of each request's first row: alone in its wave's block or its workgroup's part where
    # the length is a multiple of theirs, and alone behind a prefix where that is all there is
    print("attend, NaN in one key", shape, dtype, D, flush=True)
    c = _case(32, shape, D, dtype)
    st = c.st
    for r, n in enumerate(st.len):
        st.k[0, st.table[r][n // 16], 0, n % 16, 3] = math.nan
    _check(c, c.want(), [(0, 0), (0, 1)])


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_runs_of_keys_that_are_not_numbers(shape, dtype, D):
    # from the middle of a context on: some waves and workgroups see nothing else
    print("attend, NaN in many keys", shape, dtype, D, flush=True)
    c = _case(33, shape, D, dtype)
    st = c.st
    r = int(np.argmax(st.len))
    for p in range(st.len[r] // 2, st.len[r] + 1):
        st.k[0, st.table[r][p // 16], 1, p % 16, 0] = math.nan
    a = c.offsets[r] + r
    _check(c, c.want(), [(a, 2), (a, 3)])


@pytest.mark.parametrize("dtype,D,rows", [("bf16", 128, [1, 2, 1]), ("fp16", 64, [40, 70, 36]), ("bf16", 256, [40, 1, 36])])
def test_a_prefix_of_keys_that_are_not_numbers(dtype, D, rows):
    # the group's part is NaN throughout, the requests' own keys are finite
    print("attend, NaN prefix", dtype, D, rows, flush=True)
    c = Case(34, [144, 150, 40], rows, 4, 2, D, dtype, 16, groups=[(2, 9)])
    for p in range(144):
        c.st.k[0, c.shared[0][p // 16], 1, p % 16, 5] = math.nan
    _check(c, c.want(), [(0, 2), (0, 3), (rows[0], 2)])


@pytest.mark.parametrize("rows,groups", [([1, 3, 2], []), ([40, 70, 36], []), ([1, 2, 1], [(2, 1)]), ([40, 36, 70], [(2, 1)])])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_infinite_scores(rows, groups, dtype, D):
    # an infinite key: +inf for some rows, whose result is NaN, and -inf for the others, which go without it
    print("attend, infinite scores", rows, groups, dtype, D, flush=True)
    c = Case(35, [40, 20, 0], rows, 4, 2, D, dtype, 16, groups=groups)
    sign = np.where(np.arange(c.rows) % 2 == 0, -1.0, 1.0)
    c.q[:, :, 0] = cu.rounded(sign, dtype)[:, None]
    st = c.st
    for r, n in enumerate(st.len):
        st.k[0, st.table[r][n // 16], 0, n % 16, 0] = 0.0
    reach = c.want()[3]
    for r, n in enumerate(st.len):
        st.k[0, st.table[r][n // 16], 0, n % 16, 0] = math.inf
    out, lse, spread, _ = c.want()
    up = np.repeat(sign[:, None] > 0, c.H, 1) & (np.arange(c.H) < 2)[None]
    assert np.isnan(out[up]).all() and np.isfinite(out[1::2, 2:]).all()
    lse[up] = math.nan
    first = c.offsets[2] + 2  # request 2's first row sees this key alone
    alone = [(first, h) for h in (0, 1) if sign[first] < 0]
    for t, h in alone:
        out[t, h], spread[t, h], lse[t, h] = 0.0, 0.0, -math.inf
    c.check(want=(out, lse, spread, reach))
