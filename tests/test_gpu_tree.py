"""GPU parity of drafted trees' bookkeeping (merge, plan, acceptance, the path's K and V)
against the oracle, whole numbers and copied values bit for bit."""
import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from oracle import cache as oc
from oracle import tree as ot

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _full(*shape, value=-7, dtype=torch.int32):
    return torch.full(shape, value, dtype=dtype, device=cu.DEV)


def _status():
    return _full(1, value=0)


def signed(words):
    """Words of 64 bits as int64 holds them."""
    return [w - (1 << 64) if w >> 63 else w for w in words]


def forest(rng, n, most=4, roots=0.0):
    """Parents of a request's n nodes."""
    return [-1 if j == 0 or rng.random() < roots else int(rng.integers(max(0, j - most), j)) for j in range(n)]


@pytest.mark.parametrize("R,S,K,V", [(1, 1, 1, 2), (3, 9, 7, 2), (5, 63, 1, 40), (7, 1, 63, 3), (130, 4, 7, 5), (1000, 3, 5, 1000),
                                     (8192, 2, 2, 3),
                                     (16, 9, 7, 2), (17, 4, 7, 3), (32, 21, 3, 2), (33, 3, 15, 2),
                                     (64, 7, 9, 2), (65, 4, 3, 2)])  # one workgroup takes up to 64
def test_merge(R, S, K, V):
    _say("merge", R, S, K, V)
    rng = np.random.default_rng(R + S)
    chains = rng.integers(-1, V, (R, S, K))  # few tokens: many beginnings are equal
    for lens in (None, rng.integers(-1 if R == 7 else 0, K + (2 if R == 7 else 1), (R, S))):
        counts, offsets, drafts, parent = _full(R), _full(R + 1), _full(R * S * K), _full(R * S * K + R)
        status = _status()
        B.dspark_tree_merge(cu.i32(chains.reshape(R * S, K)), None if lens is None else cu.i32(lens.reshape(-1)), S, counts, offsets,
                            drafts, parent, status)
        torch.cuda.synchronize()
        w = ot.merge(chains.tolist(), (np.full((R, S), K) if lens is None else lens).tolist())
        n = w[1][-1]
        assert counts.tolist() == w[0] and offsets.tolist() == w[1] and int(status.item()) == w[4]
        assert drafts.tolist() == w[2] + [-7] * (R * S * K - n)
        assert parent.tolist() == w[3] + [-7] * (R * S * K - n)


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("sizes,roots", [([1], 0.0), ([64, 0, 3, 33], 0.0), ([1, 63, 64, 2, 17] * 9, 0.1)])
def test_plan(sizes, roots, lead):
    _say("plan", sizes[:5], roots, lead)
    rng = np.random.default_rng(len(sizes))
    sizes = [max(n, lead) for n in sizes]
    parent = sum((forest(rng, n, roots=roots) for n in sizes), []) + [0, 0]
    offsets = np.concatenate([[0], np.cumsum(np.array(sizes) - lead)]).tolist()
    n = len(parent)
    depth, anc, status = _full(n), _full(n, dtype=torch.int64), _status()
    B.dspark_tree_plan(cu.i32(parent), cu.i32(offsets), lead, 64, depth, anc, status)
    torch.cuda.synchronize()
    wd, wa = [-7] * n, [-7] * n
    assert ot.plan(parent, offsets, lead, 64, wd, wa) == int(status.item()) == 0
    assert depth.tolist() == wd and anc.tolist() == [x if x < 0 else signed([x])[0] for x in wa]


def test_plan_flags_what_is_no_tree():
    _say("plan, bad parents and offsets")
    parent = [-1, 0, 2, 2, -1, 4, 5, -2, -1, 1, 0, -1, 7, 1 << 30, 0, -(1 << 31), 0, 3]
    for offsets in ([0, 7, 12], [0, 60, 12], [0, 17, 3], [-1, 7, 12], [0, 7, 2_000_000_000]):
        n, R = len(parent), len(offsets) - 1
        depth, anc, status = _full(n), _full(n, dtype=torch.int64), _status()
        B.dspark_tree_plan(cu.i32(parent), cu.i32(offsets), 1, 40, depth, anc, status)
        torch.cuda.synchronize()
        wd, wa = [-7] * n, [-7] * n
        assert ot.plan(parent, offsets, 1, 40, wd, wa) == int(status.item()) == B.STATUS_BAD_ROW, R
        assert depth.tolist() == wd and anc.tolist() == wa


def _accept(drafts, offsets, parent, target, K, out=True):
    R = len(offsets) - 1
    a, path, nxt, said, status = _full(R), _full(R, K), _full(R), _full(R, K + 1), _status()
    B.dspark_accept_tree(cu.i32(drafts), cu.i32(offsets), cu.i32(parent), cu.i32(target), a, path, nxt, said if out else None, status)
    torch.cuda.synchronize()
    return a.tolist(), path.tolist(), nxt.tolist(), said.tolist(), int(status.item())


@pytest.mark.parametrize("R,most,K", [(1, 1, 0), (9, 63, 63), (100, 20, 5), (300, 63, 7)])
def test_accept(R, most, K):
    _say("accept", R, most, K)
    rng = np.random.default_rng(R)
    sizes = [int(n) for n in rng.integers(0, most + 1, R)]
    offsets = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    parent = sum((forest(rng, n + 1, most=3) for n in sizes), [])
    # few tokens: long paths, and siblings that say the same
    drafts, target = rng.integers(0, 2, sum(sizes)).tolist(), rng.integers(0, 2, sum(sizes) + R).tolist()
    want = ot.accept(drafts, offsets, parent, target, K)
    assert _accept(drafts, offsets, parent, target, K) == want
    assert K == 0 or max(want[0]) > 0
    assert _accept(drafts, offsets, parent, target, K, out=False)[:3] == want[:3]


def test_accept_of_a_chain_is_accept_greedy():
    _say("accept, chains")
    rng = np.random.default_rng(4)
    R, K = 70, 15
    sizes = rng.integers(0, K + 1, R)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    drafts, target = rng.integers(0, 2, R * K), rng.integers(0, 2, R * K + R)
    parent = sum((list(range(-1, n)) for n in sizes.tolist()), []) + [0] * (R * K - int(sizes.sum()))
    got = _accept(drafts, offsets, parent, target, K)
    a, nxt, said = _full(R), _full(R), _full(R, K + 1)
    B.dspark_accept_greedy(cu.i32(drafts), cu.i32(offsets), cu.i32(target), R, K, a, nxt, said)
    torch.cuda.synchronize()
    assert (got[0], got[2], got[3]) == (a.tolist(), nxt.tolist(), said.tolist())


def test_accept_flags_bad_rows_and_ends():
    _say("accept, bad rows")
    # a node that is its own parent, one before its parent, and offsets that fall, pass the end or hold 64 drafts
    parent, target = [-1, 1, 3, 0, 0] + [0] * 75, [5, 5, 5, 5, 5] + [5] * 75
    drafts = [5] * 70
    for offsets in ([0, 4], [0, 4, 2, 9], [0, 71], [-1, 3], [0, 64], [0, 63], [0, 2_000_000_000]):
        R = len(offsets) - 1
        assert _accept(drafts, offsets, (parent + [0] * R)[:70 + R], (target + [5] * R)[:70 + R], 5) == \
            ot.accept(drafts, offsets, (parent + [0] * R)[:70 + R], (target + [5] * R)[:70 + R], 5)


def _state(seed, page, layers, heads, D, dtype, lens, nodes):
    rng = np.random.default_rng(seed)
    need = [0 if n < 0 else -(-(n + m) // page) for n, m in zip(lens, nodes)]
    st = cu.State(rng, layers, sum(need) + 3, page, heads, D, dtype, len(lens), max(need) + 1, fill=0.0)
    st.len = list(lens)
    for r, n in enumerate(need):
        st.give(r, n)
    for x in (st.k, st.v):
        x[:] = cu.rounded(rng.standard_normal(x.shape), dtype).double().numpy()
    st.upload()
    return st, rng


def _ways(rng, nodes, K, lead=1):
    path, accept = [], []
    for n in nodes:
        many = int(rng.integers(0, min(K, n - lead) + 1))
        way = sorted(rng.choice(np.arange(lead, n), many, replace=False).tolist())
        path.append(way + [-1] * (K - many))
        accept.append(many)
    return path, accept


@pytest.mark.parametrize("page,layers,heads,D,dtype", [(16, 1, 1, 64, "bf16"), (64, 3, 2, 128, "fp16"), (256, 2, 5, 256, "bf16"),
                                                       (16, 4, 8, 128, "bf16")])
@pytest.mark.parametrize("lead", [0, 1])
def test_keep_path(page, layers, heads, D, dtype, lead):
    _say("keep path", page, layers, heads, D, dtype, lead)
    lens, nodes = [0, 3, 15, -1, 16, 250, 31, 7], [64, 1, 40, 9, 64, 20, 2, 33]
    st, rng = _state(page + D, page, layers, heads, D, dtype, lens, nodes)
    for K in (63, 4):
        path, accept = _ways(rng, nodes, K, lead)
        granted = [1, 1, 0, 1, 1, 1, 1, 1] if K == 4 else None
        status = _status()
        B.dspark_cache_keep_path(st.cache, cu.i32(path), cu.i32(accept), lead, granted=None if granted is None else cu.i32(granted),
                                 status=status)
        torch.cuda.synchronize()
        assert ot.keep_path(st.k, st.v, st.table, st.len, st.ref, path, accept, lead, granted) == int(status.item()) == 0
        st.assert_data()
        st.assert_books()


def test_keep_path_leaves_out_what_does_not_fit():
    _say("keep path, bad rows")
    lens, nodes = [10] * 9, [60] * 9
    st, rng = _state(3, 16, 2, 2, 64, "bf16", lens, nodes)
    good = [3, 9, 30, 59]
    path = [good] * 9
    path[1] = [3, 3, 30, 59]        # does not rise
    path[2] = [0, 9, 30, 59]        # from before the first draft on
    path[3] = [3, 9, 30, 64]        # past the most nodes
    path[4] = [3, 9, 30, 63]        # fits, in a page that is not there
    accept = [4, 4, 4, 4, 4, 5, -1, 4, 4]
    st.ref[st.table[7][0]] = 2      # what the path goes to is another row's too
    st.ref[st.table[8][4]] = 2      # ... and where it only comes from
    st.len[0] = 2_000_000_000
    st.upload()
    for bits, rows in ((ot.BAD_ROW, (0, 1, 2, 3, 5, 6)), (ot.BAD_PAGE, (4, 7)), (0, (8,))):
        keep = [1 if r in rows else 0 for r in range(9)]
        status = _status()
        B.dspark_cache_keep_path(st.cache, cu.i32(path), cu.i32(accept), 1, granted=cu.i32(keep), status=status)
        torch.cuda.synchronize()
        assert ot.keep_path(st.k, st.v, st.table, st.len, st.ref, path, accept, 1, keep) == int(status.item()) == bits
        st.assert_data()


def test_keep_path_past_32_bits():
    # pages whose elements, and whose layers, are numbered past 2^32
    _say("keep path, large")
    layers, page, heads, D, n_pages = 3, 256, 8, 256, 6000
    c = B.PagedCache(layers, n_pages, page, heads, D, B.DSPARK_BF16, 1, 2, device=cu.DEV)
    assert c.k.numel() > 1 << 33
    c.table.copy_(cu.i32([[n_pages - 1, n_pages - 2]]))
    c.len.fill_(240)
    c.ref[n_pages - 2:] = 1
    for i, x in enumerate((c.k, c.v)):
        x[:, n_pages - 2:] = torch.randn(x[:, n_pages - 2:].shape, generator=torch.Generator(device=cu.DEV).manual_seed(i), device=cu.DEV).to(x.dtype)
    tail = [x[:, n_pages - 2:].cpu().double().numpy() for x in (c.k, c.v)]
    k, v = oc.unpack_k(tail[0]), oc.unpack_v(tail[1])
    status, path = _status(), [[2, 17, 40]]
    B.dspark_cache_keep_path(c, cu.i32(path), cu.i32([3]), 1, status=status)
    torch.cuda.synchronize()
    assert ot.keep_path(k, v, [[1, 0]], [240], [1, 1], path, [3], 1) == int(status.item()) == 0
    np.testing.assert_array_equal(oc.unpack_k(c.k[:, n_pages - 2:].cpu().double().numpy()), k)
    np.testing.assert_array_equal(oc.unpack_v(c.v[:, n_pages - 2:].cpu().double().numpy()), v)
    assert not c.k[:, :n_pages - 2].any()
