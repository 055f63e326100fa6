"""GPU parity of the paged cache's bookkeeping (reserve, trim, commit, fork, compact) and of
append against the oracle, whole numbers and copied values bit for bit, alone and in the
order in which serving steps use them."""

import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from confidence_scheduled_verification_amd import inputs
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=cu.DEV)


def _books(seed, rows, width, n_pages, page=16, fill=0.6, layers=1, heads=1, D=64, dtype="bf16", data=False):
    """A state whose rows hold random pages (about `fill` of them in all), some rows vacant or empty."""
    rng = np.random.default_rng(seed)
    st = cu.State(rng, layers, n_pages, page, heads, D, dtype, rows, width, fill=0.0)
    for r in range(rows):
        kind = rng.random()
        if kind < 0.1:
            st.len[r] = -1
        elif kind < 0.2:
            st.len[r] = 0
        else:
            left = sum(n == 0 for n in st.ref)
            pages = int(min(rng.integers(0, width + 1), max(0, left - (1 - fill) * n_pages)))
            st.give(r, pages)
            held = sum(p >= 0 for p in st.table[r])
            st.len[r] = int(rng.integers(max(0, (held - 2) * page), held * page + 1))
    if data:
        for x in (st.k, st.v):
            x[:] = cu.rounded(rng.standard_normal(x.shape), dtype).double().numpy()
    st.upload()
    return st, rng


@pytest.mark.parametrize("rows,width,n_pages,fill", [(1, 1, 1, 1.0), (5, 4, 30, 0.5), (64, 9, 300, 0.9), (300, 70, 9000, 0.95),
                                                      (1000, 5, 20000, 0.1), (8192, 3, 24000, 0.9)])
def test_reserve(rows, width, n_pages, fill):
    _say("reserve", rows, width, n_pages, fill)
    st, rng = _books(rows, rows, width, n_pages, fill=fill)
    ws = B.pages_workspace(st.cache, rows)
    for lead, most in ((1, 7), (0, 60), (1, 16 * width)):
        offsets = np.concatenate([[0], np.cumsum(rng.integers(0, most + 1, rows))]).tolist()
        granted, status = torch.full((rows,), -7, dtype=torch.int32, device=cu.DEV), _status()
        ws.fill_(-1)
        B.dspark_pages_reserve(st.cache, cu.i32(offsets), lead, granted, ws, status)
        torch.cuda.synchronize()
        w, ws_ = oc.reserve(st.table, st.len, st.ref, offsets, lead, 16)
        np.testing.assert_array_equal(granted.cpu().numpy(), w)
        assert int(status.item()) == ws_
        st.assert_books()


def test_reserve_refuses_rows_without_their_pages():
    _say("reserve bad rows")
    st, _ = _books(3, 6, 4, 40, fill=0.3)
    for r in range(6):
        st.len[r] = 20
    st.table[0] = [-1] * 4            # says 20 tokens, holds none
    st.len[1] = 2_000_000_000         # more than a table holds
    st.upload()
    offsets = [0, 3, 6, 9, 4, 40, 2_000_000_000]   # a falling one, and one that fits no table
    granted, status = torch.zeros(6, dtype=torch.int32, device=cu.DEV), _status()
    B.dspark_pages_reserve(st.cache, cu.i32(offsets), 1, granted, B.pages_workspace(st.cache, 6), status)
    torch.cuda.synchronize()
    w, ws_ = oc.reserve(st.table, st.len, st.ref, offsets, 1, 16)
    np.testing.assert_array_equal(granted.cpu().numpy(), w)
    assert int(status.item()) == ws_ and w[0] == w[1] == 0
    st.assert_books()


@pytest.mark.parametrize("rows,width,n_pages", [(1, 1, 3), (7, 5, 60), (300, 130, 9000)])
def test_trim(rows, width, n_pages):
    _say("trim", rows, width, n_pages)
    st, rng = _books(rows + 1, rows, width, n_pages)
    keep = rng.integers(-1, 16 * width + 40, rows).tolist()
    status = _status()
    B.dspark_pages_trim(st.cache, None, cu.i32(keep), status)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.trim(st.table, st.len, st.ref, range(rows), keep, 16) == 0
    st.assert_books()
    # a list of rows, some named twice or not rows at all
    rows_ = rng.integers(-1, rows + 1, rows + 3).tolist() + [rows - 1, rows - 1]
    keep = rng.integers(-1, 16 * width, len(rows_)).tolist()
    B.dspark_pages_trim(st.cache, cu.i32(rows_), cu.i32(keep), status)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.trim(st.table, st.len, st.ref, rows_, keep, 16)
    st.assert_books()
    B.dspark_pages_trim(st.cache)  # everything freed
    torch.cuda.synchronize()
    oc.trim(st.table, st.len, st.ref, range(rows), [0] * rows, 16)
    st.assert_books()
    assert not any(st.ref)


def test_trim_flags_pages_that_nobody_holds():
    _say("trim bad pages")
    st, _ = _books(5, 4, 3, 20, fill=0.2)
    st.table = [[1, 25, -1], [2, -1, -1], [3, 3, -1], [-1] * 3]
    st.ref = [0] * 20
    st.ref[1] = st.ref[3] = 1
    st.upload()
    status = _status()
    B.dspark_pages_trim(st.cache, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.STATUS_BAD_PAGE
    assert not st.cache.ref.any() and (st.cache.table == -1).all()


def test_commit():
    _say("commit")
    st, rng = _books(8, 40, 12, 400, fill=0.9)
    accept = rng.integers(-1, 40, 40).tolist()
    accept[3] = 2_000_000_000
    status = _status()
    B.dspark_pages_commit(st.cache, cu.i32(accept), 1, status)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.commit(st.table, st.len, st.ref, accept, 1, 16)
    st.assert_books()


@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("rows,width,n_pages,fill,layers,heads,D,dtype,page",
                         [(9, 4, 60, 0.4, 2, 1, 64, "bf16", 16), (40, 7, 300, 0.5, 3, 2, 128, "fp16", 32),
                          (30, 12, 5000, 0.05, 1, 1, 256, "bf16", 16), (64, 5, 150, 0.9, 1, 3, 64, "fp16", 16)])
def test_fork(deep, rows, width, n_pages, fill, layers, heads, D, dtype, page):
    _say("fork", deep, rows, width, n_pages, fill, layers, heads, D, dtype, page)
    st, rng = _books(rows, rows, width, n_pages, page, fill, layers, heads, D, dtype, data=True)
    ws = B.pages_workspace(st.cache, 2 * rows)
    for _ in range(2):
        empty = [r for r in range(rows) if st.table[r][0] < 0]
        n = max(1, len(empty))
        dst = (rng.permutation(empty).tolist() or [0]) + rng.integers(-1, rows + 1, 4).tolist()
        src = rng.integers(0, rows, n).tolist() + rng.integers(-1, rows + 1, 4).tolist()
        dst.append(dst[0])
        src.append(src[0])
        forked, status = torch.full((len(src),), -7, dtype=torch.int32, device=cu.DEV), _status()
        ws.fill_(-1)
        B.dspark_pages_fork(st.cache, cu.i32(src), cu.i32(dst), forked, ws, deep=deep, status=status)
        torch.cuda.synchronize()
        w, st_, pairs = oc.fork(st.table, st.len, st.ref, src, dst, deep, page)
        for a, b in pairs:
            st.k[:, b], st.v[:, b] = st.k[:, a], st.v[:, a]
        np.testing.assert_array_equal(forked.cpu().numpy(), w)
        assert int(status.item()) == st_
        st.assert_books()
        st.assert_data()
        oc.trim(st.table, st.len, st.ref, dst[:n // 2], [0] * (n // 2), page)
        st.upload()


def test_many_forks_of_one_parent():
    _say("fork, many")
    rows = 2050
    st, _ = _books(1, rows, 3, 2200, fill=0.0, data=True)
    st.table[7], st.len, st.ref[9], st.ref[11] = [9, 11, -1], [0] * rows, 1, 1
    st.table = [[-1] * 3 if r != 7 else st.table[7] for r in range(rows)]
    st.ref = [int(p in (9, 11)) for p in range(2200)]
    st.len[7] = 20
    st.upload()
    dst = [r for r in range(rows) if r != 7]
    src = [7] * len(dst)
    forked = torch.zeros(len(dst), dtype=torch.int32, device=cu.DEV)
    B.dspark_pages_fork(st.cache, cu.i32(src), cu.i32(dst), forked, B.pages_workspace(st.cache, len(dst)))
    torch.cuda.synchronize()
    w, _, pairs = oc.fork(st.table, st.len, st.ref, src, dst, False, 16)
    for a, b in pairs:
        st.k[:, b], st.v[:, b] = st.k[:, a], st.v[:, a]
    np.testing.assert_array_equal(forked.cpu().numpy(), w)
    st.assert_books()
    st.assert_data()


@pytest.mark.parametrize("rows,width,n_pages,fill,layers,heads,D,dtype,page",
                         [(1, 1, 1, 1.0, 1, 1, 64, "bf16", 16), (9, 4, 60, 0.4, 2, 1, 64, "bf16", 16),
                          (40, 7, 300, 0.5, 3, 2, 128, "fp16", 32), (300, 40, 9000, 0.6, 1, 1, 64, "bf16", 16),
                          (30, 12, 5000, 0.05, 1, 1, 64, "fp16", 16), (5, 6, 20, 0.0, 1, 1, 64, "fp16", 16)])
def test_compact(rows, width, n_pages, fill, layers, heads, D, dtype, page):
    _say("compact", rows, width, n_pages, fill, layers, heads, D, dtype, page)
    st, rng = _books(rows, rows, width, n_pages, page, fill, layers, heads, D, dtype, data=True)
    if n_pages > 20:  # a page held by several rows, and one that no row holds but the caller
        full = [r for r in range(rows) if st.table[r][0] >= 0]
        st.table[full[0]][0] = st.table[full[-1]][0]
        st.ref = [sum(row.count(p) for row in st.table) for p in range(n_pages)]
        st.ref[n_pages - 1] += 1
    st.upload()
    ws = B.pages_workspace(st.cache, 0)
    ws.fill_(-1)
    page_map = torch.full((n_pages,), -7, dtype=torch.int32, device=cu.DEV)
    n_live, status = torch.zeros(1, dtype=torch.int32, device=cu.DEV), _status()
    B.dspark_pages_compact(st.cache, page_map, n_live, ws, status)
    torch.cuda.synchronize()
    w_map, w_live, w_st, moves = oc.compact(st.table, st.ref)
    for a, b in moves:
        st.k[:, b], st.v[:, b] = st.k[:, a], st.v[:, a]
    np.testing.assert_array_equal(page_map.cpu().numpy(), w_map)
    assert int(n_live.item()) == w_live and int(status.item()) == w_st
    st.assert_books()
    st.assert_data()


def test_compact_clears_entries_without_a_page():
    _say("compact bad entries")
    st, _ = _books(5, 3, 3, 20, fill=0.2)
    st.table, st.ref = [[4, 9, -1], [50, 4, -1], [-1] * 3], [0] * 20
    st.ref[4] = 2
    st.upload()
    page_map, n_live, status = (torch.zeros(n, dtype=torch.int32, device=cu.DEV) for n in (20, 1, 1))
    B.dspark_pages_compact(st.cache, page_map, n_live, B.pages_workspace(st.cache, 0), status)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.compact(st.table, st.ref)[2] == B.STATUS_BAD_PAGE
    st.assert_books()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,D,page", [(1, 64, 16), (3, 128, 32), (2, 256, 128)])
def test_append(heads, D, page, dtype):
    _say("append", heads, D, page, dtype)
    rng = np.random.default_rng(D)
    lens, rows = [0, 1, 15, 16, -1, 40, 130, 31], [1, 16, 1, 17, 3, 50, 200, 0]
    width = -(-340 // page) + 1
    st = cu.State(rng, 2, 8 * width, page, heads, D, dtype, 8, width)
    for r in range(8):
        st.len[r] = lens[r]
        if lens[r] >= 0:
            st.give(r, -(-(lens[r] + rows[r]) // page))
            st.put(1, st.table[r], 0, lens[r])
    st.upload()
    offsets, n = np.concatenate([[0], np.cumsum(rows)]).tolist(), sum(rows)
    wide = cu.rounded(rng.standard_normal((n + 2, (2 * heads + 1) * D)), dtype).to(cu.DEV)
    kn, vn = wide[:, D:(1 + heads) * D].unflatten(1, (heads, D)), wide[:, (1 + heads) * D:].unflatten(1, (heads, D))
    status = _status()
    B.dspark_cache_append(st.cache, 1, kn, vn, cu.i32(offsets), 0, 200, status)
    torch.cuda.synchronize()
    oc.append(st.k[1], st.v[1], st.table, st.len, kn.cpu().double().numpy(), vn.cpu().double().numpy(), offsets, 0)
    assert int(status.item()) == 0
    st.assert_data()
    st.assert_books()


def test_append_leaves_out_what_does_not_fit():
    _say("append bad")
    rng = np.random.default_rng(1)
    st = cu.State(rng, 1, 20, 16, 2, 64, "bf16", 4, 4)
    st.len = [10, 5, 60, 20]
    for r, n in enumerate((2, 1, 4, 2)):
        st.give(r, n)
    st.table[0][1] = -1   # the second page of request 0 was never reserved
    st.table[3][1] = 77
    st.upload()
    before = st.k.copy()
    offsets = [0, 11, 14, 30, 35]   # request 2 runs past its table
    kn = cu.rounded(rng.standard_normal((39, 2, 64)), "bf16").to(cu.DEV)
    status = _status()
    B.dspark_cache_append(st.cache, 0, kn, kn, cu.i32(offsets), 1, 20, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.STATUS_BAD_ROW | B.STATUS_BAD_PAGE
    x = kn.cpu().double().numpy()
    for r, n in ((0, 6), (1, 4)):  # what has a page is written
        a = offsets[r] + r
        for j in range(n):
            p = st.len[r] + j
            before[0, st.table[r][p // 16], :, p % 16] = x[a + j]
    np.testing.assert_array_equal(oc.unpack_k(st.cache.k.cpu().double().numpy()), before)
    status.zero_()
    B.dspark_cache_append(st.cache, 0, kn[:30], kn[:30], cu.i32(offsets), 1, 20, status)  # rows past the tensor
    B.dspark_cache_append(st.cache, 0, kn, kn, cu.i32([0, -9, 12, 30, 35]), 1, 3, status)
    torch.cuda.synchronize()
    assert int(status.item()) & B.STATUS_BAD_ROW


def test_serving_steps():
    """Steps as an engine runs them: schedule, reserve, append, attend, accept, commit, with
    forks, finished rows and a compaction between, every buffer against the oracle."""
    R, K, H, Hkv, D, page, layers, dtype = 12, 7, 8, 2, 64, 16, 2, "bf16"
    rng = np.random.default_rng(21)
    rows, width, n_pages = R + 2, 12, 150
    st = cu.State(rng, layers, n_pages, page, Hkv, D, dtype, rows, width)
    prefix = [70, 3]                                   # two pages that all requests begin with
    for p in prefix:
        st.ref[p] = R + 1                              # each row's, and the engine's own hold
    for la in range(layers):
        st.put(la, prefix, 0, 2 * page)
    for r in range(R):
        st.table[r][:2] = prefix
        st.len[r] = 2 * page
    st.len[4], st.table[4] = -1, [-1] * width          # a slot of the batch without a request
    st.ref[70] -= 1
    st.ref[3] -= 1
    c = st.upload()
    shared_row = list(prefix)
    ws, page_ws = B.cache_workspace(c, R, H, K + 1, 1), B.pages_workspace(c, rows)
    w = inputs.WORKLOADS["small"]
    vc = torch.from_numpy(B.dspark_force_monotone(inputs.raw_verify_cost(w, None))).to(cu.DEV)
    dc = torch.from_numpy(B.dspark_force_monotone(inputs.raw_draft_cost(w))).to(cu.DEV)
    for step in range(7):
        _say("serving step", step)
        status = _status()
        conf = torch.from_numpy(rng.random((R, K)).astype(np.float32)).to(cu.DEV)
        toks = cu.i32(rng.integers(0, 50, (R, K)))
        out = B.StepBuffers(R, K)
        B.dspark_schedule(conf, R, 0, R, vc, dc, out, tokens=toks, status=status)
        granted = torch.zeros(R, dtype=torch.int32, device=cu.DEV)
        B.dspark_pages_reserve(c, out.offsets, 1, granted, page_ws, status)
        n = R * (K + 1)
        q = torch.randn((layers, n, H, D), device=cu.DEV).to(torch.bfloat16)
        kv = torch.randn((layers, 2, n, Hkv, D), device=cu.DEV).to(torch.bfloat16)
        res = torch.zeros((layers, n, H, D), dtype=torch.bfloat16, device=cu.DEV)
        shared = (cu.i32([0, R]), cu.i32([shared_row]), cu.i32([2]))
        for la in range(layers):
            B.dspark_cache_append(c, la, kv[la, 0], kv[la, 1], out.offsets, 1, K + 1, status)
            B.dspark_cache_attend(c, la, q[la], out.offsets, 1, K + 1, 0.125, res[la], shared=shared, ws=ws, status=status)
        target = out.ver_tokens.new_zeros(n)
        target.copy_(cu.i32(rng.integers(0, 2, n)))    # some drafts match by chance
        accept, bonus = torch.zeros(R, dtype=torch.int32, device=cu.DEV), torch.zeros(R, dtype=torch.int32, device=cu.DEV)
        B.dspark_accept_greedy(out.ver_tokens, out.offsets, target, R, K, accept, bonus, status=status)
        B.dspark_pages_commit(c, accept, 1, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        off = out.offsets.cpu().tolist()
        g, _ = oc.reserve(st.table, st.len, st.ref, off, 1, page)
        assert granted.cpu().tolist() == g == [int(r != 4) for r in range(R)]
        for la in range(layers):
            x = kv[la].cpu().double().numpy()
            oc.append(st.k[la], st.v[la], st.table, st.len, x[0], x[1], off, 1)
            want = oc.attend(q[la].cpu().double().numpy(), st.k[la], st.v[la], st.table, st.len, off, 1, 0.125)
            cu.assert_attend(res[la], None, want, dtype, 200, D, 0.0)
        oc.commit(st.table, st.len, st.ref, accept.cpu().tolist(), 1, page)
        st.assert_books()
        st.assert_data()
        # between the steps: a request ends and another one branches into its row; parked rows
        done, parent = int(rng.integers(5, R)), int(rng.integers(0, 4))
        B.dspark_pages_trim(c, cu.i32([done, R + 1]), cu.i32([0, 0]), status)
        oc.trim(st.table, st.len, st.ref, [done, R + 1], [0, 0], page)
        forked = torch.zeros(2, dtype=torch.int32, device=cu.DEV)
        src, dst = [parent, parent], [done, R + 1]
        B.dspark_pages_fork(c, cu.i32(src), cu.i32(dst), forked, page_ws, deep=False, status=status)
        f, s, pairs = oc.fork(st.table, st.len, st.ref, src, dst, False, page)
        if step % 3 == 2:
            page_map, n_live = torch.zeros(n_pages, dtype=torch.int32, device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
            B.dspark_pages_compact(c, page_map, n_live, page_ws, status)
            m, _, _, moves = oc.compact(st.table, st.ref)
            pairs = pairs + moves
            shared_row = page_map[torch.tensor(shared_row, device=cu.DEV).long()].tolist()
            assert shared_row == st.table[0][:2]
        torch.cuda.synchronize()
        for a, b in pairs:
            st.k[:, b], st.v[:, b] = st.k[:, a], st.v[:, a]
        assert forked.cpu().tolist() == f and int(status.item()) == s == 0
        st.assert_books()
        st.assert_data()


def test_bookkeeping_in_a_captured_graph():
    _say("books in a graph")
    st, rng = _books(2, 20, 8, 200, fill=0.5)
    ws = B.pages_workspace(st.cache, 20)
    offsets = np.concatenate([[0], np.cumsum(rng.integers(0, 8, 20))]).tolist()
    off, keep = cu.i32(offsets), cu.i32(st.len)
    granted = torch.zeros(20, dtype=torch.int32, device=cu.DEV)

    def step():
        B.dspark_pages_trim(st.cache, None, keep)
        B.dspark_pages_reserve(st.cache, off, 1, granted, ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
    oc.trim(st.table, st.len, st.ref, range(20), list(st.len), 16)
    w, _ = oc.reserve(st.table, st.len, st.ref, offsets, 1, 16)
    np.testing.assert_array_equal(granted.cpu().numpy(), w)
    st.assert_books()


def test_a_shared_page_is_not_written_to():
    # a fork cut back into a page that its parent holds too: its tokens are left out
    _say("append to a shared page")
    rng = np.random.default_rng(23)
    st = cu.State(rng, 1, 8, 16, 1, 64, "bf16", 2, 4)
    st.len = [40, -1]
    st.give(0, 3)
    st.put(0, st.table[0], 0, 48)
    c = st.upload()
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    ws, flag = B.pages_workspace(c, 2), torch.zeros(2, dtype=torch.int32, device=cu.DEV)
    B.dspark_pages_fork(c, cu.i32([0]), cu.i32([1]), flag[:1], ws, status=status)
    B.dspark_pages_trim(c, cu.i32([1]), cu.i32([20]), status=status)
    offsets = cu.i32([0, 0, 3])
    B.dspark_pages_reserve(c, offsets, 0, flag, ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    before = c.k.clone(), c.v.clone()
    kn = torch.ones((3, 1, 64), dtype=torch.bfloat16, device=cu.DEV)
    B.dspark_cache_append(c, 0, kn, kn, offsets, 0, 3, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.STATUS_BAD_PAGE
    for a, b in zip(before, (c.k, c.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_refused_requests_are_not_committed():
    # a step in which one request's rows pass its table and another one's find no pages, while the
    # acceptance counted their (meaningless) tokens: both stay as they were, the others go on
    _say("commit, refused requests")
    rng = np.random.default_rng(61)
    R, page, width, lead = 5, 16, 10, 1
    st = cu.State(rng, 1, 22, page, 2, 64, "bf16", R, width)
    st.len = [155, 30, 33, -1, 20]
    for r, n in enumerate((10, 2, 3, 0, 2)):
        st.give(r, n)
        st.put(0, st.table[r], 0, max(st.len[r], 0))
    c = st.upload()
    rows = [8, 5, 100, 2, 12]
    offsets = np.concatenate([[0], np.cumsum(np.asarray(rows) - lead)]).tolist()
    off, n = cu.i32(offsets), sum(rows)
    granted, status = torch.zeros(R, dtype=torch.int32, device=cu.DEV), _status()
    ws = B.pages_workspace(c, R)
    B.dspark_pages_reserve(c, off, lead, granted, ws, status)
    kv = torch.randn((2, n, 2, 64), device=cu.DEV).to(torch.bfloat16)
    B.dspark_cache_append(c, 0, kv[0], kv[1], off, lead, max(rows), status)
    torch.cuda.synchronize()
    want, w_st = oc.reserve(st.table, st.len, st.ref, offsets, lead, page)
    assert want == [0, 1, 0, 0, 1] == granted.cpu().tolist() and w_st == B.STATUS_NO_PAGES
    status.zero_()
    accept = [4, 2, 7, 0, 11]   # requests 0 and 2 have room for as many
    B.dspark_pages_commit(c, cu.i32(accept), lead, status, granted=granted)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.commit(st.table, st.len, st.ref, accept, lead, page, want) == 0
    assert st.len == [155, 33, 33, -1, 32]
    st.assert_books()
    accept = [3, -1, 2_000_000_000, 5, 60]   # a refused request's count is not looked at
    B.dspark_pages_commit(c, cu.i32(accept), lead, status, granted=granted)
    torch.cuda.synchronize()
    assert int(status.item()) == oc.commit(st.table, st.len, st.ref, accept, lead, page, want) == B.STATUS_BAD_ROW
    st.assert_books()


def test_steps_of_a_cache_that_runs_out():
    # reserve and commit step after step in a captured graph, with granted handed on, until most
    # requests are refused
    _say("books, running out")
    st, rng = _books(62, 24, 6, 90, fill=0.8)
    R = 24
    off, accept = cu.i32([0] * (R + 1)), cu.i32([0] * R)
    granted, status, ws = torch.zeros(R, dtype=torch.int32, device=cu.DEV), _status(), B.pages_workspace(st.cache, R)

    def step():
        B.dspark_pages_reserve(st.cache, off, 1, granted, ws, status)
        B.dspark_pages_commit(st.cache, accept, 1, status, granted=granted)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g_, _ = oc.reserve(st.table, st.len, st.ref, [0] * (R + 1), 1, 16)
    oc.commit(st.table, st.len, st.ref, [0] * R, 1, 16, g_)
    st.assert_books()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    refused = 0
    for _ in range(8):
        drafts = rng.integers(0, 8, R)
        offsets, acc = np.concatenate([[0], np.cumsum(drafts)]).tolist(), [int(rng.integers(0, d + 1)) for d in drafts]
        off.copy_(cu.i32(offsets))
        accept.copy_(cu.i32(acc))
        status.zero_()
        g.replay()
        torch.cuda.synchronize()
        g_, s0 = oc.reserve(st.table, st.len, st.ref, offsets, 1, 16)
        s1 = oc.commit(st.table, st.len, st.ref, acc, 1, 16, g_)
        assert granted.cpu().tolist() == g_ and int(status.item()) == s0 | s1
        st.assert_books()
        refused += sum(not x and n >= 0 for x, n in zip(g_, st.len))
    assert refused
