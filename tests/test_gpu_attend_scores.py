"""Attention over the paged cache where scores are not finite: a NaN in a query or in a key
that a row sees makes that row's result with the key's heads NaN, whichever form computes it,
however its keys are split over waves and workgroups, and behind a shared prefix.  The
oracle (64 bits) gives NaN there by itself; all other rows and heads keep their bounds."""
import math

import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("rows,lens,groups", [([1, 1], [600, 40], []), ([70, 40], [600, 33], []),
                                              ([2, 1], [608, 600], [(2, 37)]), ([40, 70], [608, 600], [(2, 37)])])
@pytest.mark.parametrize("dtype,D", [("fp16", 64), ("fp16", 128), ("fp16", 256), ("bf16", 128)])
def test_many_small_weights_beside_a_large_one(rows, lens, groups, dtype, D):
    """The first key outweighs each other one by 2^26, and its value is zero, so that the result is
    the others' alone.  A weight of 2^-26 is below fp16's smallest number, 2^-24, and half of it;
    the kernels scale fp16 weights by 2^6, so that the rounding of each is off by at most
    half of 2^-24, 2^-31 of the largest weight (a bf16 weight by 2^-8 of itself)."""
    print("attend, small weights", rows, lens, groups, dtype, D, flush=True)
    c = Case(36, lens, rows, 2, 1, D, dtype, 16, groups=groups)
    st = c.st
    c.scale, value = 0.125, 1000.0
    c.q.zero_()
    c.q[:, :, 1] = 12.0
    for r, n in enumerate(lens):
        for p in range(n + rows[r]):
            at = (0, st.table[r][p // 16], slice(None), p % 16)
            st.k[at], st.v[at] = 0.0, value if p else 0.0
            if p == 0:
                st.k[at + (1,)] = 12.0
    out, lse, spread, reach = c.want()
    keys = max(lens) + max(rows)
    p = c.prepared()
    c.call(p)
    assert out.max() > 0.9 * value * max(lens) * math.exp(-18.0)
    off = np.abs(p["out"].cpu().double().numpy() - out)
    # e: the score's and exp2's roundings (18 is exact in either type); the sums' of up to `keys` terms
    rel = 2 * (2.0 ** -24 * 4 * 26 + 2.0 ** -21) + 2 * keys * 2.0 ** -24
    step = 2.0 ** -8 * out if dtype == "bf16" else keys * 2.0 ** -31 * value
    bound = 1.05 * (step + rel * out) + out * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -11) + 2.0 ** -25
    assert int(p["status"].item()) == 0 and (off <= bound).all(), (off.max(), bound.max(), out.max())
    assert (np.abs(p["lse"].cpu().double().numpy() - lse) <= rel + 2.0 ** -22 * np.abs(lse)).all()


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D,size", [("bf16", 128, 1e5), ("fp16", 64, 4e3), ("bf16", 256, 1e15), ("fp16", 128, 4e3)])
def test_very_large_finite_scores(shape, dtype, D, size):
    """Scores so large that a rounding of one is many powers of two: the largest still has a
    weight of one, and where it leads by far the result is its value."""
    print("attend, large scores", shape, dtype, D, flush=True)
    c = _case(37, shape, D, dtype)
    c.q = cu.rounded(c.q.double().numpy() * size, dtype)
    k = c.st.k[0]
    k[np.isfinite(k)] *= size
    c.st.k[0] = cu.rounded(k, dtype).double().numpy()
    out, lse, _, reach = c.want()
    p = c.prepared()
    c.call(p)
    got, got_lse = p["out"].cpu().double().numpy(), p["lse"].cpu().double().numpy()
    assert int(p["status"].item()) == 0 and np.isfinite(got).all() and np.isfinite(got_lse).all()
    # scores and lse are off by at most (D + 8) 2^-24 of the largest sum of |q||k|; where the second
    # score lies behind by more than twice that, and by 40, its weight is below every rounding, and
    # what is left are the roundings of the one weight and of the result, half a step each, and exp2's
    err = (D + 8) * 2.0 ** -24 * reach
    assert (np.abs(got_lse - lse) <= 1.05 * err + 2.0 ** -22 * np.abs(lse) + 2.0 ** -20).all()
    first, second = _two_largest(c)
    clear = first - second > 2 * err + 40
    assert clear.mean() > 0.5
    half = float(torch.finfo(cu.DT[dtype][1]).eps) / 2
    off = np.abs(got - out)[clear]
    assert (off <= 1.05 * (2 * half + 2.0 ** -21) * np.abs(out)[clear] + 2.0 ** -25).all(), off.max()


def _two_largest(c):
    """Each (row, head)'s two largest scores, -inf where there is no second key."""
    st, q = c.st, c.q.double().numpy()
    G, two = c.H // st.k.shape[2], np.full((2, c.rows, c.H), -math.inf)
    for r, n in enumerate(st.len):
        a, b = c.offsets[r] + r, c.offsets[r + 1] + r + 1
        pos = np.arange(n + b - a)
        ids = np.array(st.table[r])[pos // c.page]
        for t in range(a, b):
            for h in range(c.H):
                s = np.sort(c.scale * (st.k[0][ids, h // G, pos % c.page][:n + 1 + t - a] @ q[t, h]))
                two[:s[-2:].size, t, h] = s[::-1][:2]
    return two
