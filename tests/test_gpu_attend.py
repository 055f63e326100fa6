"""GPU parity of the paged cache's attention (dspark_cache_attend) against the oracle in 64
bits: key heads and groups of heads, dims, page sizes and types, ragged and vacant
requests, shared prefixes, values that are not numbers in masked places, bad tables,
strides, long contexts split over the device, and a captured call replayed."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


class Case:
    """Requests over a cache: lens (-1: vacant) and rows per request, behind shared pages of
    `groups` (a list of (requests, pages))."""

    def __init__(self, seed, lens, rows, H, Hkv, D, dtype="bf16", page=16, lead=1, groups=(), layers=1, layer=0, extra=3,
                 pad=0):
        rng = np.random.default_rng(seed)
        R = len(lens)
        self.lead, self.layer, self.H, self.D, self.dtype, self.page = lead, layer, H, D, dtype, page
        need = [0 if n < 0 else -(-(n + m) // page) for n, m in zip(lens, rows)]
        width = max(1, max(need) + 1)
        n_pages = sum(need) + sum(p for _, p in groups) + extra
        self.st = st = cu.State(rng, layers, n_pages, page, Hkv, D, dtype, R, width)
        st.len = list(lens)
        self.group_off, self.shared = [0], []
        r0, of = 0, {}
        for count, pages in groups:
            free = rng.permutation([p for p, n in enumerate(st.ref) if n == 0])[:pages].tolist()
            for p in free:
                st.ref[p] = count + 1
            st.put(layer, free, 0, pages * page)
            self.shared.append(free)
            for r in range(r0, r0 + count):
                of[r] = free
            r0 += count
            self.group_off.append(r0)
        for r in range(R):
            if lens[r] < 0:
                continue
            own = need[r] - len(of.get(r, []))
            free = rng.permutation([p for p, n in enumerate(st.ref) if n == 0])[:own].tolist()
            for p in free:
                st.ref[p] = 1
            ids = of.get(r, []) + free
            st.table[r][:len(ids)] = ids
            first = len(of.get(r, [])) * page
            st.put(layer, ids, first, lens[r] + rows[r] - first)
        self.offsets = np.concatenate([[0], np.cumsum(np.asarray(rows) - lead)]).astype(int).tolist()
        self.rows = sum(rows) + pad
        self.max_new = max(rows)
        self.q = cu.rounded(rng.standard_normal((self.rows, H, D)), dtype)
        self.scale = 1.0 / math.sqrt(D)

    def want(self, upto=None):
        st = self.st
        n = sum(1 for _ in self.offsets) - 1
        return oc.attend(self.q.double().numpy(), st.k[self.layer], st.v[self.layer], st.table[:n], st.len, self.offsets,
                         self.lead, self.scale)

    def prepared(self, max_new=None):
        c = self.st.upload()
        self.left = 7.0
        q = self.q.to(cu.DEV)
        out = torch.full((self.rows, self.H, self.D), self.left, dtype=q.dtype, device=cu.DEV)
        lse = torch.full((self.rows, self.H), self.left, dtype=torch.float32, device=cu.DEV)
        shared = None
        if self.shared:
            w = max(1, max(len(s) for s in self.shared))
            table = np.full((len(self.shared), w), -1)
            for i, s in enumerate(self.shared):
                table[i, :len(s)] = s
            shared = (cu.i32(self.group_off), cu.i32(table), cu.i32([len(s) for s in self.shared]))
        status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
        self.max_new = max_new or self.max_new
        ws = B.cache_workspace(c, len(self.offsets) - 1, self.H, self.max_new, len(self.shared))
        ws.fill_(0x7FC00000)  # nothing in a workspace is counted on: NaN, or counts beyond every bound
        return dict(q=q, out=out, lse=lse, shared=shared, status=status, ws=ws, offsets=cu.i32(self.offsets))

    def call(self, p, **kw):
        B.dspark_cache_attend(self.st.cache, self.layer, kw.get("q", p["q"]), p["offsets"], self.lead, self.max_new,
                              self.scale, kw.get("out", p["out"]), lse=kw.get("lse", p["lse"]), shared=p["shared"],
                              ws=p["ws"], status=p["status"])

    def check(self, status=0, max_new=None, want=None):
        p = self.prepared(max_new)
        self.call(p)
        torch.cuda.synchronize()
        assert int(p["status"].item()) == status
        keys = max(max(self.st.len), 0) + self.max_new
        cu.assert_attend(p["out"], p["lse"], want or self.want(), self.dtype, keys, self.D, self.left)
        return p


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hkv,page", [(1, 1, 16), (6, 2, 16), (8, 8, 32), (40, 1, 128)])
def test_single_and_few_rows(D, dtype, H, Hkv, page):
    _say("attend", D, dtype, H, Hkv, page)
    Case(D + H, [0, 1, 15, 16, 17, 31, 127, 128, 300], [1, 1, 1, 2, 1, 4, 1, 3, 8], H, Hkv, D, dtype, page).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,H,Hkv,page", [(128, 8, 2, 16), (64, 3, 3, 64), (256, 4, 1, 32)])
def test_prompts(D, H, Hkv, page, dtype):
    _say("attend prompts", D, H, Hkv, page, dtype)
    Case(5, [0, 40, 7, 0], [70, 1, 129, 0], H, Hkv, D, dtype, page, lead=0).check()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
@pytest.mark.parametrize("groups", [[(6, 9)], [(2, 3), (4, 17)], [(3, 0), (1, 20)], [(0, 4), (5, 1)]])
def test_shared_prefixes(groups, dtype, D):
    _say("attend shared", groups, dtype, D)
    sh = [p for n, p in groups for _ in range(n)]
    own = [0, 33, 1, 250, 16, 5]
    lens = [(sh[r] * 16 if r < len(sh) else 0) + own[r] for r in range(6)]
    Case(9, lens, [3, 1, 8, 2, 5, 8], 8, 2, D, dtype, 16, groups=groups).check()


@pytest.mark.parametrize("groups", [[(20, 12)], [(7, 5), (13, 30)]])
def test_shared_prefix_of_many_rows(groups):
    # more rows of a group than a tile holds, so that the groups' part has many tiles
    _say("attend shared, many rows", groups)
    sh = [p for n, p in groups for _ in range(n)]
    rng = np.random.default_rng(3)
    lens = [s * 16 + int(x) for s, x in zip(sh, rng.integers(0, 60, 20))]
    rows = rng.integers(1, 9, 20).tolist()
    for dtype, D, H, Hkv in (("bf16", 128, 10, 2), ("fp16", 64, 4, 4), ("bf16", 256, 8, 1)):
        Case(4, lens, rows, H, Hkv, D, dtype, 16, groups=groups).check()


def test_vacant_requests_and_rows_of_nobody():
    _say("attend vacant")
    p = Case(2, [-1, 20, -1, 64, -5], [2, 1, 1, 3, 8], 4, 2, 64, pad=5).check()
    assert (p["out"][:2] == 0).all() and torch.isneginf(p["lse"][:2]).all()
    Case(2, [-1, -1], [2, 1], 4, 2, 128).check()
    c = Case(2, [-1, 40, -1, 32], [2, 1, 1, 2], 4, 2, 128, groups=[(4, 2)])  # in a group too
    c.check()


def test_rows_beyond_the_bound_are_left_alone():
    _say("attend max_new")
    c = Case(8, [30, 5, 18], [2, 7, 1], 4, 1, 64)
    want = list(c.want())
    a, b = oc.rows_of(c.offsets, 1, 1)
    want[3][a:b] = -1  # rows of nobody
    c.check(status=B.STATUS_BAD_ROW, max_new=4, want=want)


@pytest.mark.parametrize("special", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_masked_values_have_no_say(special, dtype):
    # the last rows' own keys and values are not numbers: earlier rows see none of it
    _say("attend special", special, dtype)
    c = Case(6, [10, 130, 16], [4, 8, 1], 4, 2, 64, dtype)
    st = c.st
    for r, j in ((0, 2), (1, 5)):
        p = st.len[r] + j
        st.v[0, st.table[r][p // 16], 0, p % 16, 3:20] = special
        st.v[0, st.table[r][p // 16], 1, p % 16, 60] = special
        if math.isnan(special):
            st.k[0, st.table[r][p // 16], 1, p % 16, 0] = special
    p = st.len[1] + 6  # and one of the other sign
    st.v[0, st.table[1][p // 16], 0, p % 16, 5] = -special
    want = c.want()
    assert np.isfinite(want[0][:2]).all() and not np.isfinite(want[0][2:4]).all()
    c.check(want=want)


def test_empty_calls_write_nothing():
    _say("attend empty")
    c = Case(1, [4], [1], 2, 2, 64)
    p = c.prepared()
    e = p["q"][:0]
    B.dspark_cache_attend(c.st.cache, 0, e, p["offsets"], 1, 1, 1.0, e.clone(), ws=p["ws"])
    B.dspark_cache_attend(c.st.cache, 0, p["q"], p["offsets"][:1], 1, 1, 1.0, p["out"], ws=p["ws"])
    B.dspark_cache_attend(c.st.cache, 0, p["q"], p["offsets"], 0, 0, 1.0, p["out"], ws=p["ws"])
    torch.cuda.synchronize()
    assert (p["out"] == 7).all()


def test_bad_tables_and_lengths_are_flagged():
    _say("attend bad tables")
    for bad_id in (-1, 1 << 30, -(1 << 31)):
        c = Case(3, [50, 20, 40], [2, 1, 3], 4, 2, 128)
        c.st.table[0][1] = bad_id  # tokens 16..31 of request 0 are not there
        c.check(status=B.STATUS_BAD_PAGE)
    c = Case(3, [50, 20, 40], [2, 1, 3], 4, 2, 128)  # a length beyond the table: the request sees nothing
    want = list(c.want())
    c.st.len[0] = 2_000_000_000
    for w in want:
        w[:2] = 0
    want[1][:2] = -np.inf
    p = c.prepared()
    c.call(p)
    torch.cuda.synchronize()
    assert int(p["status"].item()) == B.STATUS_BAD_ROW
    cu.assert_attend(p["out"], p["lse"], want, "bf16", 50, 128, 7.0)


def test_bad_offsets_are_left_out():
    _say("attend bad offsets")
    c = Case(3, [50, 20, 40], [2, 1, 3], 4, 2, 64)
    p = c.prepared()
    for off in ([1 << 30, 1, 1, 3], [0, -5, 1, 3], [0, 1, 1 << 30, 3], [-2, 1, 1, 3]):
        p["offsets"].copy_(cu.i32(off))
        p["status"].zero_()
        c.call(p)
        torch.cuda.synchronize()
        assert int(p["status"].item()) & B.STATUS_BAD_ROW


def test_bad_groups_are_flagged():
    _say("attend bad groups")
    c = Case(3, [50, 34, 40], [2, 1, 3], 4, 2, 64, groups=[(3, 2)])
    c.check()
    p = c.prepared()
    for off, pages, want in (([0, 9], [2], B.STATUS_BAD_ROW), ([2, 1], [2], B.STATUS_BAD_ROW), ([0, 3], [5], B.STATUS_BAD_ROW),
                             ([0, 3], [-1], B.STATUS_BAD_ROW), ([-4, 3], [2], B.STATUS_BAD_ROW)):
        p["shared"][0].copy_(cu.i32(off))
        p["shared"][2].copy_(cu.i32(pages))
        p["status"].zero_()
        c.call(p)
        torch.cuda.synchronize()
        assert int(p["status"].item()) & want, (off, pages)
    c = Case(3, [50, 34, 40], [2, 1, 3], 4, 2, 64, groups=[(3, 2)])
    c.st.table[1][0] = c.st.table[0][3]  # not the group's page: flagged, the group's counts
    p = c.prepared()
    c.call(p)
    torch.cuda.synchronize()
    assert int(p["status"].item()) == B.STATUS_BAD_PAGE


def test_row_strides_and_no_lse():
    _say("attend strides")
    c = Case(7, [90, 3, 260], [5, 1, 2], 6, 3, 128)
    p = c.prepared()
    H, D = c.H, c.D
    wide = torch.randn((c.rows, (H + 6) * D), device=cu.DEV).to(p["q"].dtype)
    q = wide[:, 3 * D:(3 + H) * D].unflatten(1, (H, D))
    q.copy_(p["q"])
    wide_out = torch.full((c.rows, H * D + 24), 7.0, dtype=q.dtype, device=cu.DEV)
    out = wide_out[:, 8:8 + H * D].unflatten(1, (H, D))
    c.call(p, q=q, out=out, lse=None)
    torch.cuda.synchronize()
    cu.assert_attend(out, None, c.want(), "bf16", 270, D)
    assert (wide_out[:, :8] == 7).all() and (wide_out[:, 8 + H * D:] == 7).all()


@pytest.mark.parametrize("R,ctx,groups", [(1, 20000, []), (3, 5001, []), (2, 6400, [(2, 300)])])
def test_long_contexts_are_split_and_joined(R, ctx, groups):
    # one head pair's keys over many workgroups; checked against float64 on the host
    _say("attend long", R, ctx, groups)
    lens = [ctx - 77 * r for r in range(R)]
    Case(11, lens, [2] * R, 4, 2, 64, "bf16", 16, groups=groups).check()


def test_layers_and_pages_past_32_bits():
    # the last pages of a cache of over 2^32 elements a tensor, in its second layer
    _say("attend 64-bit offsets")
    D, Hkv, page = 256, 8, 128
    n_pages = (1 << 31) // (D * Hkv * page) + 70   # a layer's elements pass 2^31, two pass 2^32
    st = B.PagedCache(2, n_pages, page, Hkv, D, B.DSPARK_BF16, 2, 4, device=cu.DEV)
    rng = np.random.default_rng(0)
    table, lens, offsets = [[n_pages - 1, n_pages - 3, -1, -1], [0, n_pages - 2, -1, -1]], [150, 130], [0, 1, 1]
    st.table.copy_(cu.i32(table))
    st.len.copy_(cu.i32(lens))
    kn = cu.rounded(rng.standard_normal((3, Hkv, D)), "bf16")
    vn = cu.rounded(rng.standard_normal((3, Hkv, D)), "bf16")
    ids = [n_pages - 1, n_pages - 3, 0, n_pages - 2]
    local = cu.rounded(rng.standard_normal((2, 4, Hkv, page, D)), "bf16")
    st.k[1, ids] = torch.from_numpy(oc.pack_k(local[0].float().numpy())).to(cu.DEV).bfloat16()
    st.v[1, ids] = torch.from_numpy(oc.pack_v(local[1].float().numpy())).to(cu.DEV).bfloat16()
    B.dspark_cache_append(st, 1, kn.to(cu.DEV), vn.to(cu.DEV), cu.i32(offsets), 1, 2)
    k, v = local.double().numpy()
    small = [[0, 1], [2, 3]]
    oc.append(k, v, small, lens, kn.double().numpy(), vn.double().numpy(), offsets, 1)
    q = cu.rounded(rng.standard_normal((3, Hkv, D)), "bf16")
    out = torch.empty((3, Hkv, D), dtype=torch.bfloat16, device=cu.DEV)
    B.dspark_cache_attend(st, 1, q.to(cu.DEV), cu.i32(offsets), 1, 2, 0.0625, out, ws=B.cache_workspace(st, 2, Hkv, 2))
    torch.cuda.synchronize()
    cu.assert_attend(out, None, oc.attend(q.double().numpy(), k, v, small, lens, offsets, 1, 0.0625), "bf16", 152, D)
    assert not st.k[0, ids].any()


def test_many_requests():
    # as many requests as a call takes, most of them vacant or single tokens
    _say("attend many requests")
    R = 8192
    rng = np.random.default_rng(1)
    lens = np.where(rng.random(R) < 0.97, -1, rng.integers(0, 40, R)).tolist()
    Case(12, lens, [1] * R, 2, 1, 64).check()


def test_determinism_and_a_captured_call():
    _say("attend graph")
    c = Case(13, [1200, 30, -1, 700, 9], [3, 8, 1, 1, 2], 8, 2, 128, groups=[(2, 1)])
    c.check()
    p = c.prepared()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.call(p)
    s.synchronize()
    first, first_lse = p["out"].clone(), p["lse"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(p)
    q0 = p["q"].clone()
    for i in range(4):
        p["q"].copy_(q0 * (1 if i % 2 == 0 else -1))
        p["out"].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        if i % 2 == 0:
            assert torch.equal(p["out"], first) and torch.equal(p["lse"], first_lse)
        else:
            assert not torch.equal(p["out"], first)
        eager = torch.full_like(p["out"], 7.0)
        c.call(p, out=eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, p["out"])


# Requests and groups of more than 64 columns, which the kernels bring to LDS for all waves.

@pytest.mark.parametrize("special", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256), ("fp16", 128)])
def test_masked_values_have_no_say_in_prompts(special, dtype, D):
    # values that are not numbers early, at a stage's end and in the last row's own place: rows
    # before them see none of it, rows from there on all of it
    _say("attend special, prompts", special, dtype, D)
    c = Case(16, [10, 130, 0], [90, 75, 130], 4, 2, D, dtype)
    st = c.st
    for r, j, head in ((0, 3, 0), (0, 89, 1), (1, 62, 0), (2, 127, 1), (2, 64, 0)):
        p = st.len[r] + j
        st.v[0, st.table[r][p // 16], head, p % 16, 3:20] = special
        st.v[0, st.table[r][p // 16], head, p % 16, D - 1] = -special
    if math.isnan(special):
        p = st.len[1] + 50
        st.k[0, st.table[1][p // 16], 1, p % 16, 0] = special
    want = c.want()
    assert np.isfinite(want[0][:3]).all() and np.isfinite(want[0][165:165 + 64]).all()
    assert not np.isfinite(want[0][3]).all() and not np.isfinite(want[0][-1]).all()
    c.check(want=want)


@pytest.mark.parametrize("special", [math.nan, math.inf])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_special_values_in_a_shared_prefix(special, dtype, D):
    # a prefix that ends inside a stage of 64, with one such value near its start and one near its end
    _say("attend special, prefix", special, dtype, D)
    c = Case(17, [9 * 16 + 5] * 12, [8] * 12, 4, 2, D, dtype, groups=[(6, 9), (6, 9)])
    st = c.st
    for g, p in ((0, 3), (0, 140)):
        st.v[0, c.shared[g][p // 16], 1, p % 16, 7:9] = special
    want = c.want()
    assert not np.isfinite(want[0][:48]).all() and np.isfinite(want[0][48:]).all()
    c.check(want=want)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256)])
def test_bad_pages_of_prompts_and_prefixes(dtype, D):
    # pages that are not there in the middle and at the ends: their tokens are left out
    _say("attend bad pages, many rows", dtype, D)
    for bad_id in (-1, 1 << 30, -(1 << 31)):
        c = Case(18, [200, 20], [80, 100], 4, 2, D, dtype)
        for r, i in ((0, 0), (0, 5), (0, 6), (0, 7), (0, 8), (1, 2)):
            c.st.table[r][i] = bad_id
        c.check(status=B.STATUS_BAD_PAGE)
    c = Case(18, [13 * 16 + 9] * 20, [8] * 20, 4, 2, D, dtype, groups=[(20, 13)])
    for r in range(20):
        c.st.table[r][4] = c.st.table[r][12] = -1
    c.shared[0][4] = c.shared[0][12] = -1
    c.check(status=B.STATUS_BAD_PAGE)


@pytest.mark.parametrize("rows,lens", [([64, 1, 0, 65], [0, 300, 12, 63]), ([16, 17], [64, 0]), ([300], [0]), ([129, 2, 128], [-1, 5, 1])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_prompts(rows, lens, D):
    # tiles and stages that end early, requests with none of the other's columns, vacant ones
    _say("attend ragged prompts", rows, lens, D)
    Case(19, lens, rows, 4, 1, D, "bf16", 64, lead=0, pad=3).check()


def test_long_context_of_many_columns():
    # more than 64 stages of 64 keys to a workgroup, against float64 on the device
    _say("attend long, many columns")
    D, Hkv, H, page, T, rows = 128, 8, 64, 16, 150001, 9
    n_pages = -(-(T + rows) // page)
    st = B.PagedCache(1, n_pages + 2, page, Hkv, D, B.DSPARK_BF16, 1, n_pages, device=cu.DEV)
    g = torch.Generator(device=cu.DEV).manual_seed(5)
    st.k.normal_(generator=g)
    st.v.normal_(generator=g)
    ids = torch.randperm(n_pages + 2, generator=g, device=cu.DEV)[:n_pages]
    st.table[0] = ids.to(torch.int32)
    st.len.fill_(T)
    q = torch.randn((rows, H, D), generator=g, device=cu.DEV).bfloat16()
    out, lse = torch.empty_like(q), torch.empty((rows, H), device=cu.DEV)
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    scale = 1 / math.sqrt(D)
    B.dspark_cache_attend(st, 0, q, cu.i32([0, rows - 1]), 1, rows, scale, out, lse=lse,
                          ws=B.cache_workspace(st, 1, H, rows), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = [np.empty((rows, H, D)), np.empty((rows, H)), np.empty((rows, H, D)), np.empty((rows, H))]
    last = T + torch.arange(rows, device=cu.DEV)
    for h in range(Hkv):
        k = st.k[0, ids, h, 0].double().permute(0, 2, 1, 3).reshape(-1, D)
        v = st.v[0, ids, h, 0].double().permute(0, 2, 1).reshape(-1, D)
        hs = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
        x = q[:, hs].double().reshape(-1, D)
        s = scale * torch.mm(x, k.t().contiguous())
        s.masked_fill_(torch.arange(k.shape[0], device=cu.DEV)[None] > last.repeat_interleave(H // Hkv)[:, None], -math.inf)
        l = torch.logsumexp(s, 1)
        w = torch.exp(s - l[:, None])
        reach = scale * torch.mm(x.abs(), k.abs().t().contiguous()).amax(1)
        for i, y in enumerate((torch.mm(w, v), l, torch.mm(w, v.abs()), reach)):
            want[i][:, hs] = y.reshape((rows, H // Hkv) + tuple(y.shape[1:])).cpu().numpy()
    cu.assert_attend(out, lse, want, "bf16", T + rows, D)


def test_two_captured_calls_share_a_workspace():
    _say("attend two graphs, one workspace")
    a = Case(20, [70, 90, 33], [40, 8, 30], 4, 2, 128, groups=[(2, 3)])
    b = Case(21, [700, -1, 9], [2, 1, 8], 8, 2, 64, "fp16")
    pa, pb = a.prepared(), b.prepared()
    if pb["ws"].numel() > pa["ws"].numel():
        pa["ws"] = pb["ws"]
    else:
        pb["ws"] = pa["ws"]
    s, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(s):
        a.call(pa)
        b.call(pb)
    s.synchronize()
    want = [pa["out"].clone(), pb["out"].clone()]
    for c, p in ((a, pa), (b, pb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(p)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0)):
        pa["out"].fill_(7.0)
        pb["out"].fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(pa["out"], want[0]) and torch.equal(pb["out"], want[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_requests_of_many_columns(D):
    # the running units of as many requests as a call takes, beside the keys in LDS
    _say("attend many requests, many columns", D)
    R = 8192
    rng = np.random.default_rng(2)
    lens = np.where(rng.random(R) < 0.99, -1, rng.integers(0, 40, R)).tolist()
    rows = [1] * R
    lens[5], rows[5], lens[8000], rows[8000] = 100, 40, 3, 37
    Case(22, lens, rows, 2, 1, D).check()


def test_offsets_that_fall_and_rise_past_all_bounds():
    # requests, then groups, that all name the same rows: more units than 32 bits number
    _say("attend falling offsets")
    R, n, page, width = 8192, 4096, 256, 4200
    st = B.PagedCache(1, 2, page, 1, 64, B.DSPARK_BF16, R, width, device=cu.DEV)
    st.table.zero_()
    st.len.fill_(width * page - n)
    q = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device=cu.DEV)
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    B.dspark_cache_attend(st, 0, q, cu.i32(np.arange(R + 1) % 2 * n), 0, n, 1.0, out, ws=B.cache_workspace(st, R, 1, n),
                          status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.STATUS_BAD_ROW and (out == 7).all()
    groups, pages = 1024, 16500
    st.len.fill_(-1)
    q = torch.zeros((R, 1, 64), dtype=torch.bfloat16, device=cu.DEV)
    out = torch.full_like(q, 7.0)
    shared = (cu.i32(np.arange(groups + 1) % 2 * R), torch.zeros((groups, pages), dtype=torch.int32, device=cu.DEV),
              cu.i32([pages] * groups))
    status.zero_()
    B.dspark_cache_attend(st, 0, q, cu.i32(np.arange(R + 1)), 0, 1, 1.0, out, shared=shared,
                          ws=B.cache_workspace(st, R, 1, 1, groups), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.STATUS_BAD_ROW and (out == 0).all()
