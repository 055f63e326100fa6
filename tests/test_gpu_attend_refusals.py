"""What attention over the paged cache leaves in every row when some requests or groups of a
call do not fit: rows of left-out requests untouched, zeros where a request sees nothing,
and the right result for all others, also beside a request of their group that is left out
and where the group itself is refused (they then read their own tables)."""

import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from oracle import cache as oc
from test_gpu_attend import Case

pytestmark = pytest.mark.gpu


def _want(c, offsets, max_new, n_rows):
    """The oracle's results request by request: those whose rows do not fit are rows of nobody,
    and a length past the table makes zeros."""
    st, R = c.st, len(offsets) - 1
    q = c.q.double().numpy()
    none = oc.attend(q, st.k[0], st.v[0], [], [], [0], 0, c.scale)
    for r in range(R):
        n, start = offsets[r + 1] - offsets[r] + c.lead, offsets[r] + c.lead * r
        if offsets[r] < 0 or not 0 < n <= max_new or start + n > min(n_rows, R * max_new):
            continue
        ln = st.len[r] if st.len[r] + n <= len(st.table[r]) * c.page else -1
        part = oc.attend(q, st.k[0], st.v[0], [st.table[r]], [ln], [start, start + n], 0, c.scale)
        for w, x in zip(none, part):
            w[start:start + n] = x[start:start + n]
    return none


def _run(c, p, offsets, status, n_rows=None, max_new=None, group_off=None, shared_pages=None):
    n_rows, c.max_new = n_rows or c.rows, max_new or c.max_new
    p["offsets"].copy_(cu.i32(offsets))
    if group_off is not None:
        p["shared"][0].copy_(cu.i32(group_off))
    if shared_pages is not None:
        p["shared"][2].copy_(cu.i32(shared_pages))
    p["status"].zero_()
    p["out"].fill_(c.left)
    p["lse"].fill_(c.left)
    p["ws"].fill_(0x7FC00000)
    B.dspark_cache_attend(c.st.cache, 0, p["q"][:n_rows], p["offsets"], c.lead, c.max_new, c.scale, p["out"][:n_rows],
                          lse=p["lse"][:n_rows], shared=p["shared"], ws=p["ws"], status=p["status"])
    torch.cuda.synchronize()
    assert int(p["status"].item()) == status
    want = _want(c, offsets, c.max_new, n_rows)
    cu.assert_attend(p["out"], p["lse"], want, c.dtype, max(max(c.st.len), 0) + c.max_new, c.D, c.left)
    return want


GROUPS = [[], [(3, 2)]]


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("rows", [[2, 1, 3], [40, 33, 50]])
def test_rows_of_bad_offsets(rows, groups):
    print("attend, bad offsets, values", rows, groups, flush=True)
    c = Case(41, [50, 34, 40], rows, 4, 2, 64, groups=groups)
    p, good = c.prepared(), c.offsets
    _run(c, p, good, 0)
    last = c.rows - 3
    for off in ([1 << 30] + good[1:], [0, -5] + good[2:], [0, good[1], 1 << 30, good[3]], [-2] + good[1:],
                [0, good[1], good[2], good[3] + 40], [good[1] + 1, 0, good[2], good[3]], [last, last - 1, 0, 0]):
        _run(c, p, off, B.STATUS_BAD_ROW)


@pytest.mark.parametrize("D,rows,max_new", [(64, [3, 6], 4), (128, [3, 6, 2], 4), (128, [40, 90, 50], 60), (256, [40, 90], 60)])
def test_a_request_beside_one_that_is_left_out(D, rows, max_new):
    # one group over all: a neighbour with too many rows, then one whose rows pass the tensor
    print("attend, a neighbour left out", D, rows, max_new, flush=True)
    R = len(rows)
    c = Case(42, [40, 64, 33][:R], rows, 4, 2, D, groups=[(R, 2)])
    p = c.prepared()
    w = _run(c, p, c.offsets, B.STATUS_BAD_ROW, max_new=max_new)
    assert np.isfinite(w[0][:rows[0]]).all() and (w[3][rows[0]:rows[0] + rows[1]] == -1).all()
    c.max_new = max(rows)
    w = _run(c, p, c.offsets, B.STATUS_BAD_ROW, n_rows=c.rows - 1)
    assert np.isfinite(w[0][:rows[0]]).all() and (w[3][-1] == -1).all()


@pytest.mark.parametrize("D,rows", [(64, [2, 1, 3]), (128, [40, 33, 50])])
def test_rows_of_groups_that_do_not_fit(D, rows):
    # the requests are served from their own tables
    print("attend, bad groups, values", D, rows, flush=True)
    c = Case(43, [50, 34, 40], rows, 4, 2, D, groups=[(3, 2)])
    p = c.prepared()
    for off, pages in (([0, 9], [2]), ([2, 1], [2]), ([0, 3], [5]), ([0, 3], [-1]), ([-4, 3], [2]), ([0, 4], [2])):
        _run(c, p, c.offsets, B.STATUS_BAD_ROW, group_off=off, shared_pages=pages)
    _run(c, p, c.offsets, 0, group_off=[0, 2], shared_pages=[2])
    # a request shorter than its group's prefix sees nothing
    c.st.len[1] = 31
    c.st.cache.len.copy_(cu.i32(c.st.len))
    p["shared"][0].copy_(cu.i32([0, 3]))
    p["status"].zero_()
    c.call(p)
    torch.cuda.synchronize()
    a, b = oc.rows_of(c.offsets, 1, 1)
    assert int(p["status"].item()) == B.STATUS_BAD_ROW
    assert (p["out"][a:b] == 0).all() and torch.isneginf(p["lse"][a:b]).all()


def test_two_groups_of_which_one_does_not_fit():
    print("attend, one bad group of two", flush=True)
    for rows in ([1, 2, 1, 3], [40, 70, 1, 36]):
        c = Case(44, [50, 34, 700, 40], rows, 4, 2, 128, groups=[(2, 2), (2, 1)])
        p = c.prepared()
        _run(c, p, c.offsets, 0)
        _run(c, p, c.offsets, B.STATUS_BAD_ROW, group_off=[0, 2, 5])
        _run(c, p, c.offsets, B.STATUS_BAD_ROW, group_off=[0, 2, 4], shared_pages=[2, -3])
        _run(c, p, c.offsets, B.STATUS_BAD_ROW, group_off=[-1, 2, 4], shared_pages=[2, 1])


@pytest.mark.parametrize("page", [64, 256])
def test_large_pages_and_their_ends(page):
    # lengths on both sides of a page's end, few columns and many, behind a prefix of whole pages
    print("attend, large pages", page, flush=True)
    for rows in ([1, 2, 1, 3], [40, 70, 1, 36]):
        for groups in ([], [(3, 1)]):
            lens = [page - 1 if not groups else page, 2 * page, page + 1, 3]
            Case(45, lens, rows, 4, 2, 128, "bf16", page, groups=groups).check()


def test_a_long_bound_over_a_long_table():
    # rows and a table of a million tokens whose product is large, of which the call uses little
    print("attend, long bounds", flush=True)
    c = Case(46, [700, 40, 90], [70, 1, 130], 8, 2, 64)
    p, n = c.prepared(), 131072
    st, R = c.st, 3
    table = torch.full((R, 1 << 16), -1, dtype=torch.int32, device=cu.DEV)
    table[:, :st.cache.width] = st.cache.table
    cache = B.PagedCache(1, st.cache.n_pages, 16, 2, 64, B.DSPARK_BF16, R, 1 << 16, k=st.cache.k, v=st.cache.v, table=table,
                         len=st.cache.len, ref=st.cache.ref)
    q = torch.zeros((n, 8, 64), dtype=torch.bfloat16, device=cu.DEV)
    q[:c.rows] = p["q"]
    out = torch.full_like(q, 7.0)
    for most in (n, (1 << 31) - 1):
        out.fill_(7.0)
        B.dspark_cache_attend(cache, 0, q, p["offsets"], 1, most, c.scale, out, ws=p["ws"], status=p["status"])
        torch.cuda.synchronize()
        assert int(p["status"].item()) == 0 and (out[c.rows:] == 7).all()
        cu.assert_attend(out[:c.rows], None, c.want(), "bf16", 830, 64)


@pytest.mark.parametrize("D,rows", [(128, [1] * 11 + [300]), (64, [300] + [1] * 5), (256, [1, 90, 2])])
def test_a_workspace_of_the_rows_alone(D, rows):
    # single tokens and a prompt behind a prefix, in a workspace sized by the rows: nothing is
    # written behind it
    print("attend, workspace by rows", D, rows, flush=True)
    R = len(rows)
    c = Case(47, [40 + 3 * r for r in range(R)], rows, 4, 2, D, groups=[(R - 1, 2)])
    p = c.prepared()
    n = B.cache_workspace(c.st.cache, R, c.H, c.max_new, 1, n_rows=c.rows).numel()
    assert n < p["ws"].numel()
    p["ws"].fill_(0x7FC00000)
    whole, p["ws"] = p["ws"], p["ws"][:n]
    c.call(p)
    torch.cuda.synchronize()
    assert int(p["status"].item()) == 0 and (whole[n:] == 0x7FC00000).all()
    cu.assert_attend(p["out"], p["lse"], c.want(), c.dtype, 400, D, c.left)


def test_groups_that_have_requests_in_common():
    # group_off that fall: no group counts, whatever each one's own range is
    print("attend, overlapping groups", flush=True)
    for rows in ([1, 2, 1, 3], [40, 70, 1, 36]):
        c = Case(48, [50, 34, 700, 40], rows, 4, 2, 128, groups=[(2, 2), (1, 1), (1, 2)])
        p = c.prepared()
        _run(c, p, c.offsets, 0)
        for off in ([0, 3, 1, 4], [0, 4, 0, 4], [2, 4, 1, 3]):
            _run(c, p, c.offsets, B.STATUS_BAD_ROW, group_off=off)
