"""GPU parity of the append with rotary positions (dspark_cache_append_rotary) against the
oracle: layouts, parts of a head, scalings, far positions, trees' depths, strides, and
what is left out."""
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


class Rows:
    """A cache whose rows hold pages for the step, and the step's packed rows."""

    def __init__(self, seed, lens, rows, H, Hkv, D, dtype="bf16", page=16, lead=1, pad=2, wide=False):
        self.rng = rng = np.random.default_rng(seed)
        self.lead, self.H, self.D, self.dtype, self.page = lead, H, D, dtype, page
        need = [0 if n < 0 else -(-(n + m) // page) for n, m in zip(lens, rows)]
        self.st = st = cu.State(rng, 2, sum(need) + 3, page, Hkv, D, dtype, len(lens), max(need) + 1, fill=0.0)
        st.len = list(lens)
        for r, n in enumerate(need):
            st.give(r, n)
        for x in (st.k, st.v):
            x[:] = cu.rounded(rng.standard_normal(x.shape), dtype).double().numpy()
        st.upload()
        self.offsets = np.concatenate([[0], np.cumsum(np.asarray(rows) - lead)]).astype(int).tolist()
        self.n, self.max_new = sum(rows) + pad, max(rows)
        x = cu.rounded(rng.standard_normal((self.n, H + 2 * Hkv, D)), dtype).to(cu.DEV)  # as one projection gives them
        self.q, self.k, self.v = (y if wide else y.contiguous() for y in (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]))
        self.q_out = torch.full((self.n, H, D), 7.0, dtype=x.dtype, device=cu.DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)

    def positions(self, depth=None):
        """(packed row, request, place, position of the turn) of every row that takes part."""
        got = []
        for r, ln in enumerate(self.st.len):
            a, b = oc.rows_of(self.offsets, self.lead, r)
            got += [(a + j, r, j, ln + (j if depth is None else depth[a + j])) for j in range(b - a) if ln >= 0]
        return got

    def call(self, rot, depth=None, q=None, q_out=None, layer=1):
        B.dspark_cache_append_rotary(self.st.cache, layer, rot, self.q if q is None else q, self.q_out if q_out is None else q_out, self.k,
                                     self.v, cu.i32(self.offsets), self.lead, self.max_new,
                                     depth=None if depth is None else cu.i32(depth), status=self.status)
        torch.cuda.synchronize()

    def bound(self, want, reach):
        """How far a turned value may be off, from the roundings alone.  The angle is exact to 2^-32 turns
        (2^-29 radians) and rounded to fp32 within half a turn (2^-25 of pi: 2^-23), sines are good to two
        units (2^-22 at most), each times the factor (2^-24); two products and a sum add 3 2^-24: all in
        all below 2^-21 of |a| + |b| times the factor, and the result's rounding is half a step (fp16:
        at least half of 2^-24)."""
        u = float(torch.finfo(cu.DT[self.dtype][1]).eps) / 2
        return 2.0 ** -21 * reach + u * np.abs(want) + 2.0 ** -25

    def check(self, rot, depth=None, status=0, layer=1, ran=None):
        """`ran`: the result of a call that was made already."""
        st, at = self.st, self.positions(depth)
        if ran is None:
            self.call(rot, depth, layer=layer)
        assert int(self.status.item()) == status
        rows, pos = [x[0] for x in at], [x[3] for x in at]
        turned = [ot.rotate(x.cpu().double().numpy()[rows], pos, rot.freq, rot.dim, rot.first, rot.interleaved, rot.attention)
                  for x in (self.q, self.k)]
        got = (self.q_out if ran is None else ran).cpu().double().numpy()
        (wq, rq), (wk, rk) = turned
        bad = ~(np.abs(got[rows] - wq) <= self.bound(wq, rq))
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[rows][bad][:4], wq[bad][:4])
        rest = np.setdiff1d(np.arange(self.n), rows)
        if ran is None:
            assert (got[rest] == 7).all()
        k, v = oc.unpack_k(st.cache.k.cpu().double().numpy()), oc.unpack_v(st.cache.v.cpu().double().numpy())
        vn = self.v.cpu().double().numpy()
        wv, kept = st.v.copy(), st.k.copy()
        for i, (t, r, j, _) in enumerate(at):
            p = st.len[r] + j
            page, slot = st.table[r][p // self.page], p % self.page
            if not 0 <= page < k.shape[1] or st.ref[page] > 1:
                continue
            wv[layer, page, :, slot] = vn[t]
            bad = ~(np.abs(k[layer, page, :, slot] - wk[i]) <= self.bound(wk[i], rk[i]))
            assert not bad.any(), (t, r, j, np.argwhere(bad)[:4].tolist())
            kept[layer, page, :, slot] = k[layer, page, :, slot]
        np.testing.assert_array_equal(v, wv)
        np.testing.assert_array_equal(k, kept)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,dim,first", [(64, 64, 0), (64, 16, 8), (128, 128, 0), (128, 64, 64), (128, 48, 24), (256, 256, 0), (256, 32, 224),
                                         (256, 240, 16)])
def test_parts_and_layouts(D, dim, first, dtype, interleaved):
    _say("rotary", D, dim, first, dtype, interleaved)
    rot = B.Rotary(dim, first=first, interleaved=interleaved, attention=1.25)
    Rows(D + dim, [0, 3, 15, -1, 16, 250], [8, 1, 33, 4, 2, 17], 6, 3, D, dtype).check(rot)


@pytest.mark.parametrize("H,Hkv,page,lead,rows", [(1, 1, 16, 1, [1, 1, 1]), (40, 5, 32, 0, [200, 0, 3]), (17, 17, 256, 1, [5, 64, 2]),
                                                  (64, 8, 64, 0, [0, 0, 1])])
def test_heads_pages_and_lengths(H, Hkv, page, lead, rows):
    _say("rotary", H, Hkv, page, lead, rows)
    rot = B.Rotary(64, 500000.0, interleaved=H == 40)
    Rows(H, [7, 0, 100], rows, H, Hkv, 64, "bf16", page, lead, wide=H == 17).check(rot)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17])
def test_few_rows(most, D):
    # one to eight tokens stand side by side in a wave, and heads or parts of one beside them
    _say("rotary, few rows", most, D)
    rows = [most, 1, (most + 1) // 2, most, 0]
    Rows(most, [5, 0, 13, -1, 40], rows, 21, 7, D, "fp16" if most % 2 else "bf16", lead=0).check(B.Rotary(D, interleaved=most > 4))


@pytest.mark.parametrize("scaling", ["none", "linear", "bands", "ramp"])
def test_far_positions_and_scalings(scaling):
    # angles are as exact at the far end of a long context as at its start
    _say("rotary, far", scaling)
    rot = B.Rotary(128, 500000.0, scaling=scaling, factor=8.0, original=8192.0, low=1.0, high=32.0, attention=1.2)
    for ln in (131072 - 5, 1_000_003):
        c = Rows(3, [5], [9], 4, 2, 128, page=256)
        width = (ln + 9) // 256 + 1
        cache = B.PagedCache(1, 3, 256, 2, 128, B.DSPARK_BF16, 1, width, device=cu.DEV)
        cache.table[0, -1], cache.table[0, -2] = 1, 2  # of the kept tokens' pages only the last ones matter
        cache.ref[1:3] = 1
        cache.len.fill_(ln)
        B.dspark_cache_append_rotary(cache, 0, rot, c.q, c.q_out, c.k, c.v, cu.i32(c.offsets), 1, 9, status=c.status)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        wq, rq = ot.rotate(c.q.cpu().double().numpy()[:9], ln + np.arange(9), rot.freq, 128, 0, False, rot.attention)
        assert (np.abs(c.q_out.cpu().double().numpy()[:9] - wq) <= c.bound(wq, rq)).all()
        wk, rk = ot.rotate(c.k.cpu().double().numpy()[:9], ln + np.arange(9), rot.freq, 128, 0, False, rot.attention)
        k = oc.unpack_k(cache.k.cpu().double().numpy())[0]
        for j in range(9):
            p = ln + j
            assert (np.abs(k[int(cache.table[0, p // 256]), :, p % 256] - wk[j]) <= c.bound(wk[j], rk[j])).all()


def test_trees_turn_by_their_depth():
    _say("rotary, depth")
    c = Rows(4, [100, 31, -1, 0], [64, 9, 3, 20], 4, 2, 128)
    rng = np.random.default_rng(0)
    depth = rng.integers(0, 9, c.n).tolist()
    depth[2] = -100    # in front of the cache's tokens, at position 0
    c.check(B.Rotary(128), depth=depth)


def test_in_place_strides_streams_and_a_captured_call():
    _say("rotary, in place")
    c = Rows(5, [40, 3], [8, 30], 4, 2, 64, wide=True)
    rot = B.Rotary(32, first=16)
    before = c.q.clone()
    want = torch.full_like(before, 7.0)
    c.call(rot, q_out=want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.dspark_cache_append_rotary(c.st.cache, 1, rot, c.q, c.q, c.k, c.v, cu.i32(c.offsets), 1, c.max_new)
    s.synchronize()
    torch.cuda.synchronize()
    rows = [x[0] for x in c.positions()]
    assert torch.equal(c.q[rows], want[rows]) and torch.equal(c.q[-2:], before[-2:])
    c.q.copy_(before)
    c.check(rot, ran=want)
    off, out, graph = cu.i32(c.offsets), torch.empty_like(before), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.dspark_cache_append_rotary(c.st.cache, 1, rot, c.q, out, c.k, c.v, off, 1, c.max_new)
    for _ in range(3):
        out.fill_(7.0)
        c.st.cache.k[1] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_what_does_not_fit_is_left_out():
    _say("rotary, refusals")
    c = Rows(6, [40, 40, 40, 40, 20], [6, 6, 6, 6, 6], 4, 2, 64)
    c.st.table[1][2] = -1                      # tokens without a page: their queries turn all the same
    c.st.ref[c.st.table[2][2]] = 2             # another row's page
    c.st.len[3] = 2_000_000_000
    c.st.upload()
    st = c.st
    st.len = [n if n < 1_000_000 else -1 for n in st.len]  # (out of all tables: left out)
    c.check(B.Rotary(64), status=B.STATUS_BAD_PAGE | B.STATUS_BAD_ROW)
    for most in (6, 9):  # rows over two pages of which one is missing or another's
        c = Rows(most, [13, 13, 13, 10, 13], [6, 6, 6, most, 6], 5, 3, 128, "fp16")
        c.st.table[0][1] = c.st.table[1][0] = -1
        c.st.ref[c.st.table[2][1]] = c.st.ref[c.st.table[4][0]] = 2
        c.st.upload()
        c.check(B.Rotary(64, first=32), status=B.STATUS_BAD_PAGE)
    c = Rows(7, [10, 10, 10], [6, 6, 6], 4, 2, 64)
    c.offsets = [0, 7, 2, 2_000_000_000]       # more rows than max_new, fewer than none, past the tensors
    c.call(B.Rotary(64))
    assert int(c.status.item()) == B.STATUS_BAD_ROW and (c.q_out == 7).all()
    c.st.assert_data()


def test_a_prompt_of_more_blocks_than_a_launch_takes():
    _say("rotary, a million rows")
    n, ln, D, page = 65535 * 16 + 37, 5, 64, 256
    width = (ln + n + page - 1) // page
    cache = B.PagedCache(1, width, page, 1, D, B.DSPARK_BF16, 1, width, device=cu.DEV)
    cache.table[0] = torch.arange(width, dtype=torch.int32, device=cu.DEV).flip(0)
    cache.ref.fill_(1)
    cache.len.fill_(ln)
    g = torch.Generator(device=cu.DEV)
    g.manual_seed(8)
    q, k, v = (torch.randn((n, 1, D), generator=g, device=cu.DEV).to(torch.bfloat16) for _ in range(3))
    out, status, rot = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device=cu.DEV), B.Rotary(D)
    B.dspark_cache_append_rotary(cache, 0, rot, q, out, k, v, cu.i32([0, n]), 0, n, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    order = cache.table[0].long()
    in_v = cache.v[0, order, 0].permute(0, 1, 3, 2).reshape(-1, D)[ln:ln + n]           # blocks as [D][16]
    in_k = cache.k[0, order, 0].permute(0, 1, 3, 2, 4).reshape(-1, D)[ln:ln + n]        # blocks as [D / 8][16][8]
    assert torch.equal(in_v, v[:, 0])
    for x, y in ((q[:, 0], out[:, 0]), (k[:, 0], in_k)):  # a turn leaves each pair as long as it was, but for two roundings
        a, b = (z.float().view(n, 2, D // 2).norm(dim=1) for z in (x, y))
        assert ((a - b).abs() <= (2.0 ** -8 + 2.0 ** -18) * a).all()
    at = torch.tensor([0, 15, 16, 65535 * 16 - 6, 65535 * 16 - 5, 65535 * 16 - 4, 65535 * 16, n - 1])
    for x, y in ((q, out[:, 0]), (k, in_k)):
        want, reach = ot.rotate(x[at].cpu().double().numpy(), ln + at.numpy(), rot.freq, D, 0, False, 1.0)
        bound = 2.0 ** -21 * reach + 2.0 ** -8 * np.abs(want) + 2.0 ** -25
        assert (np.abs(y[at].cpu().double().numpy()[:, None] - want) <= bound).all()
