"""GPU parity of attention over trees' rows (dspark_cache_attend_tree) against the oracle in
64 bits: words of every kind, key heads and groups, dims, pages and types, shared prefixes,
values that are not numbers in masked places, empty rows, a captured call replayed."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from oracle import tree as ot
from test_gpu_attend import Case
from test_gpu_tree import forest, signed

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


class Tree(Case):
    """Case with a word for every row: of random trees, or as given."""

    def __init__(self, seed, lens, rows, *args, words=None, **kw):
        super().__init__(seed, lens, rows, *args, **kw)
        rng = np.random.default_rng(seed + 1)
        parent = sum((forest(rng, n) for n in rows), []) + [-1] * (self.rows - sum(rows))
        depth, anc = [0] * self.rows, [(1 << 64) - 1] * self.rows
        assert ot.plan(parent, self.offsets, self.lead, 64, depth, anc) == 0
        self.anc = anc if words is None else words(anc, rng)

    def want(self):
        st = self.st
        return ot.attend(self.q.double().numpy(), st.k[self.layer], st.v[self.layer], st.table[:len(self.offsets) - 1], st.len,
                         self.offsets, self.lead, self.scale, self.anc)

    def call(self, p, **kw):
        anc = torch.tensor(signed(self.anc), dtype=torch.int64, device=cu.DEV) if "anc" not in p else p["anc"]
        B.dspark_cache_attend_tree(self.st.cache, self.layer, kw.get("q", p["q"]), p["offsets"], self.lead, self.max_new, anc,
                                   self.scale, kw.get("out", p["out"]), lse=kw.get("lse", p["lse"]), shared=p["shared"],
                                   ws=p["ws"], status=p["status"])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hkv,page", [(1, 1, 16), (6, 2, 16), (8, 8, 32), (40, 1, 128)])
def test_trees(D, dtype, H, Hkv, page):
    _say("tree", D, dtype, H, Hkv, page)
    Tree(D + H, [0, 1, 15, 16, 63, 31, 127, 128, 300, 0], [1, 2, 64, 9, 33, 64, 1, 31, 8, 64], H, Hkv, D, dtype, page, pad=2).check()


@pytest.mark.parametrize("D,rows", [(64, 3), (128, 2), (128, 64), (256, 40)])
def test_words_of_any_kind(D, rows):
    # nothing at all, the request's tokens alone, all nodes (later ones too), single ones, bits past the
    # request's rows, and random ones
    _say("tree, words", D, rows)

    def words(anc, rng):
        kinds = [0, 1 << 63 if rows < 64 else 1, (1 << 64) - 1, 1, 1 << (rows - 1)]
        return [kinds[i % 7] if i % 7 < 5 else int(rng.integers(0, 1 << 63)) * 2 + 1 for i in range(len(anc))]
    Tree(7, [40, 0, 130, -1, 5], [rows] * 5, 4, 2, D, words=words).check()
    Tree(8, [100] * 4, [rows] * 4, 4, 1, D, "fp16", groups=[(2, 3), (2, 6)], words=words).check()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
@pytest.mark.parametrize("groups", [[(3, 5)], [(1, 2), (2, 4)], [(1, 0), (2, 1)]])
def test_shared_prefixes(groups, dtype, D):
    _say("tree, shared", groups, dtype, D)
    Tree(3, [90, 83, 200, 12, -1], [17, 64, 1, 30, 4], 8, 2, D, dtype, groups=groups).check()


def test_a_chain_is_the_causal_call():
    _say("tree, chain")
    for rows in ([1, 8, 16], [64, 40, 3]):
        c = Tree(11, [300, 17, 64], rows, 8, 2, 128, groups=[(2, 1)])
        c.anc = sum(([(2 << j) - 1 for j in range(n)] for n in rows), [])
        p = c.check()
        out, lse = torch.full_like(p["out"], 7.0), torch.full_like(p["lse"], 7.0)
        B.dspark_cache_attend(c.st.cache, 0, p["q"], p["offsets"], 1, c.max_new, c.scale, out, lse=lse, shared=p["shared"], ws=p["ws"])
        torch.cuda.synchronize()
        assert torch.equal(out, p["out"]) and torch.equal(lse, p["lse"])


@pytest.mark.parametrize("special", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows,dtype,D", [(8, "bf16", 128), (8, "fp16", 64), (64, "bf16", 128), (64, "fp16", 64), (64, "bf16", 256)])
def test_nodes_that_are_not_seen_have_no_say(special, rows, dtype, D):
    # one node's V (and another's K) is not a number: rows off its branch see none of it
    _say("tree, special", special, rows, dtype, D)
    c = Tree(16, [10, 60], [rows, rows], 4, 2, D, dtype)
    st = c.st
    for r, j in ((0, 2), (1, rows - 3)):
        p = st.len[r] + j
        st.v[0, st.table[r][p // 16], 1, p % 16, 3:20] = special
        st.v[0, st.table[r][p // 16], 1, p % 16, D - 1] = -special
    if math.isnan(special):
        p = st.len[1] + 4
        st.k[0, st.table[1][p // 16], 0, p % 16, 0] = special
    want = c.want()
    fine = np.isfinite(want[0]).all((1, 2))
    assert fine.any() and not fine.all()
    c.check(want=want)


def test_bad_offsets_lengths_and_pages():
    _say("tree, bad rows")
    c = Tree(5, [40, 40, 40, 40], [6, 6, 6, 6], 4, 2, 128)
    c.st.len[1] = 2_000_000_000   # fits no table: its rows see nothing
    c.st.table[2][1] = 1 << 30    # tokens that are not there
    st = c.st
    lens = list(st.len)
    lens[1] = -1
    want = ot.attend(c.q.double().numpy(), st.k[0], st.v[0], st.table, lens, c.offsets, 1, c.scale, c.anc)
    c.check(status=B.STATUS_BAD_ROW | B.STATUS_BAD_PAGE, want=want)
    c = Tree(5, [40, 40], [6, 6], 4, 2, 128)
    c.offsets = [0, 70, 10]  # the first request has more rows than max_new, the second fewer than none
    p = c.prepared(max_new=64)
    c.call(p)
    torch.cuda.synchronize()
    assert int(p["status"].item()) == B.STATUS_BAD_ROW and (p["out"] == 7).all() and (p["lse"] == 7).all()


@pytest.mark.parametrize("dtype,D,H,Hkv", [("bf16", 128, 16, 2), ("fp16", 64, 8, 1), ("bf16", 256, 4, 1), ("bf16", 128, 4, 4)])
def test_long_contexts(dtype, D, H, Hkv):
    # segments split over the device, against float64 on the device
    _say("tree, long", dtype, D, H, Hkv)
    page, lens, rows = 64, [40001, 9], [64, 20]
    T = sum(lens) + sum(rows)
    c = Tree(6, [1, 1], rows, H, Hkv, D, dtype, page)
    st = B.PagedCache(1, -(-T // page) + 3, page, Hkv, D, cu.DT[dtype][0], 2, -(-T // page), device=cu.DEV)
    g = torch.Generator(device=cu.DEV).manual_seed(5)
    st.k.normal_(generator=g)
    st.v.normal_(generator=g)
    ids = torch.randperm(st.n_pages, generator=g, device=cu.DEV).to(torch.int32)
    n0 = -(-(lens[0] + rows[0]) // page)
    st.table[0, :n0] = ids[:n0]
    st.table[1, 0] = ids[n0]
    st.len.copy_(cu.i32(lens))
    q = c.q.to(cu.DEV)
    out, lse, status = torch.empty_like(q), torch.empty(q.shape[:2], device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    anc = torch.tensor(signed(c.anc), dtype=torch.int64, device=cu.DEV)
    B.dspark_cache_attend_tree(st, 0, q, cu.i32(c.offsets), 1, 64, anc, c.scale, out, lse=lse, ws=B.cache_workspace(st, 2, H, 64), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = [np.empty(q.shape), np.empty(q.shape[:2]), np.empty(q.shape), np.empty(q.shape[:2])]
    for r, (a, b) in enumerate(((0, 64), (64, 84))):
        n = lens[r] + rows[r]
        pages = st.table[r, :-(-n // page)].long()
        sees = torch.ones((b - a, n), dtype=torch.bool)
        sees[:, lens[r]:] = torch.tensor([[bool(c.anc[t] >> i & 1) for i in range(b - a)] for t in range(a, b)])
        sees = sees.to(cu.DEV).repeat_interleave(H // Hkv, 0)
        for h in range(Hkv):
            k = st.k[0, pages, h].double().permute(0, 1, 3, 2, 4).reshape(-1, D)[:n].contiguous()
            v = st.v[0, pages, h].double().permute(0, 1, 3, 2).reshape(-1, D)[:n].contiguous()
            hs = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            x = q[a:b, hs].double().reshape(-1, D)
            s = (c.scale * torch.mm(x, k.t().contiguous())).masked_fill(~sees, -math.inf)
            l = torch.logsumexp(s, 1)
            w = torch.exp(s - l[:, None])
            reach = c.scale * torch.mm(x.abs(), k.abs().t().contiguous()).amax(1)
            for i, y in enumerate((torch.mm(w, v), l, torch.mm(w, v.abs()), reach)):
                want[i][a:b, hs] = y.reshape((b - a, H // Hkv) + tuple(y.shape[1:])).cpu().numpy()
    cu.assert_attend(out, lse, want, dtype, 40065, D)


def test_row_strides_streams_and_a_captured_call():
    _say("tree, captured")
    c = Tree(9, [70, 33, -1, 500], [33, 8, 4, 64], 8, 2, 128, groups=[(2, 1)])
    p = c.prepared()
    p["anc"] = torch.tensor(signed(c.anc), dtype=torch.int64, device=cu.DEV)
    wide = torch.full((c.rows, 24, 128), 7.0, dtype=torch.bfloat16, device=cu.DEV)  # q and out beside each other
    wide[:, :8] = p["q"]
    q, out = wide[:, :8], wide[:, 8:16]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(p, q=q, out=out)
    s.synchronize()
    cu.assert_attend(out, p["lse"], c.want(), "bf16", 600, 128, 7.0)
    assert (wide[:, 16:] == 7).all()
    eager = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(p, q=q, out=out)
    for _ in range(3):
        out.fill_(7.0)
        p["ws"].fill_(0x7FC00000)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def _as_a_chain(c, rows):
    """The tree's call with the words of chains, and the causal call: the same bits."""
    c.anc = sum(([(2 << j) - 1 for j in range(n)] for n in rows), [])
    p = c.check()
    out, lse = torch.full_like(p["out"], 7.0), torch.full_like(p["lse"], 7.0)
    B.dspark_cache_attend(c.st.cache, 0, p["q"], p["offsets"], 1, c.max_new, c.scale, out, lse=lse, shared=p["shared"], ws=p["ws"])
    torch.cuda.synchronize()
    assert torch.equal(out, p["out"]) and torch.equal(lse, p["lse"])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_segments_in_any_number_of_parts(dtype, D):
    # one segment of 1 to 18 units of 128 keys, most of them in as many parts: joined eight at a time, the
    # last ones four at a time
    for parts in range(1, 19):
        _say("tree, parts", dtype, D, parts)
        Tree(parts, [128 * parts - 4], [4], 4, 1, D, dtype).check()
        _as_a_chain(Tree(parts, [128 * parts - 4], [4], 4, 1, D, dtype), [4])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_long_segments_among_many_short_ones(dtype, D):
    # so many segments that they are joined four at a time, one of them in many parts
    _say("tree, many short", dtype, D)
    rng = np.random.default_rng(D)
    rows = rng.integers(1, 5, 40).tolist()
    lens = rng.integers(0, 60, 40).tolist()
    lens[7], lens[31] = 5003, 700
    Tree(31, lens, rows, 8, 8, D, dtype).check()
    _as_a_chain(Tree(32, lens, rows, 8, 8, D, dtype), rows)
    rows = [64] * 9      # and the form of many rows
    lens = [1000, 0, 31, 5, 17, 900, 2500, 64, 1]
    Tree(33, lens, rows, 16, 8, D, dtype).check()
