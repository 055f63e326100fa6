"""GPU parity of the target's choice (dspark_target_tokens) and of its history against the
oracle, whole numbers equal and processed logits bit for bit: both are rounded alike."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B
from oracle import tree as ot
from test_gpu_tree import forest, signed

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _say(*a):
    print(*a, flush=True)


def _pack(bits, words=None):
    n, V = bits.shape
    full = np.zeros((n, (words or (V + 31) // 32) * 32), bool)
    full[:, :V] = bits
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32)).to(cu.DEV)


class Step:
    """A step's rows with everything that has a say in them; parts are left out by setting them to None."""

    def __init__(self, seed, rows, V, dtype="bf16", lead=1, seen=20, biased=5, masks=3, allow=0.5, tree=True, pad=2, shift=0):
        self.rng = rng = np.random.default_rng(seed)
        self.V, self.dtype, self.lead, R = V, dtype, lead, len(rows)
        self.R, self.sizes, self.max_new = R, rows, max(max(rows), 1)
        self.offsets = np.concatenate([[0], np.cumsum(np.asarray(rows) - lead)]).astype(int).tolist()
        self.n = sum(rows) + pad
        # few different values, so that many are equal
        x = torch.from_numpy(np.round(rng.standard_normal((self.n, V)) * 8) / 4).to(DT[dtype])
        self.buffer = torch.zeros(self.n * V + 64, dtype=x.dtype, device=cu.DEV)
        self.logits = self.buffer[shift:shift + self.n * V].view(self.n, V)
        self.logits.copy_(x)
        self.history = ot.History(R, V)
        low = lambda n: np.minimum(rng.integers(0, V, n), rng.integers(0, V, n)).tolist()  # noqa: E731
        for r in range(R):
            self.history.add([low(seen)], False, [r])
            self.history.add([low(seen // 2)], True, [r])
        self.penalties = [rng.choice([0.5, 1.0, 1.1, 1.3], R), rng.choice([0.0, 0.25, 0.3, -0.5], R), rng.choice([0.0, 0.1, 0.25], R)]
        self.drafts = low(max(self.n, 1))
        self.anc = None
        if tree:
            depth, self.anc = [0] * self.n, [0] * self.n
            ot.plan(sum((forest(rng, n) for n in rows), []) + [-1] * pad, self.offsets, lead, 64, depth, self.anc)
        self.bias = None
        if biased:
            lists = [np.sort(rng.choice(V, min(V, int(rng.integers(0, biased + 1))), replace=False)).tolist() for _ in range(R)]
            self.bias = [[(v, float(np.float32(rng.standard_normal()))) for v in x] for x in lists]
        self.allowed = rng.random((masks, V)) < allow if masks else None
        self.pick = rng.integers(-1, masks, self.n).tolist() if masks else None

    def want(self):
        targets, out = {}, {}
        pen = [np.float32(x).astype(np.float64) if x is not None else None for x in self.penalties]
        on = any(x is not None for x in pen)
        for r in range(self.R):
            a, b = self.offsets[r] + self.lead * r, self.offsets[r + 1] + self.lead * (r + 1)
            for t in range(a, b):
                j = t - a
                nodes = [i for i in range(self.lead, b - a) if (self.anc[t] >> i & 1 if self.anc is not None else i <= j)]
                path = [self.drafts[self.offsets[r] + i - self.lead] for i in nodes] if on and self.drafts is not None else []
                free = None if self.allowed is None or self.pick[t] == -1 else \
                    self.allowed[self.pick[t]] if 0 <= self.pick[t] < len(self.allowed) else np.zeros(self.V, bool)
                h = self.history if on else None
                targets[t], out[t] = ot.choose(
                    self.logits[t].double().cpu().numpy(), path, h.prompt[r] if h else (), h.count[r] if h else None,
                    *(d if x is None else x[r] for x, d in zip(pen, (1.0, 0.0, 0.0))), dict(self.bias[r]) if self.bias else None, free)
        return targets, out

    def upload(self):
        i32 = cu.i32
        f32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.float32, device=cu.DEV)  # noqa: E731
        kw = dict(penalties=tuple(f32(x) for x in self.penalties))
        if self.history is not None:
            seen, count = self.history.arrays()
            self.h = B.History(self.R, self.V, seen=torch.from_numpy(seen).to(cu.DEV), count=torch.from_numpy(count).to(cu.DEV))
            kw["history"] = self.h
        if self.drafts is not None:
            kw["node_tokens"] = i32(self.drafts)
        if self.anc is not None:
            kw["anc"] = torch.tensor(signed(self.anc), dtype=torch.int64, device=cu.DEV)
        if self.bias is not None:
            kw["bias"] = (i32(np.concatenate([[0], np.cumsum([len(x) for x in self.bias])])), i32([v for x in self.bias for v, _ in x]),
                          f32([b for x in self.bias for _, b in x]))
        if self.allowed is not None:
            kw.update(allowed=_pack(self.allowed), allowed_row=i32(self.pick))
        return kw

    def prepared(self, adjusted=True, shift=0):
        self.target = torch.full((self.n,), -7, dtype=torch.int32, device=cu.DEV)
        self.out = torch.full((self.n * self.V + 64,), 7.0, dtype=DT[self.dtype], device=cu.DEV)
        self.adjusted = self.out[shift:shift + self.n * self.V].view(self.n, self.V) if adjusted else None
        self.status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
        ws = B.target_workspace(self.n, self.V)
        ws[4096:] = -1  # behind the counts nothing is counted on
        return dict(self.upload(), ws=ws, status=self.status, adjusted=self.adjusted)

    def call(self, kw):
        B.dspark_target_tokens(self.logits, cu.i32(self.offsets), self.lead, self.max_new, self.target, **kw)

    def check(self, status=0, want=None):
        want, rounded = want or self.want(), {}
        for t, y in want[1].items():
            rounded[t] = torch.from_numpy(y).float().to(DT[self.dtype]).float().numpy()
        for adjusted, shift in ((False, 0), (True, 0), (True, 1)):
            kw = self.prepared(adjusted, shift)
            self.call(kw)
            torch.cuda.synchronize()
            got = self.target.tolist()
            bad = [(t, got[t], want[0].get(t, -7)) for t in range(self.n) if got[t] != want[0].get(t, -7)]
            assert not bad, bad[:5]
            assert int(self.status.item()) == status
            if not adjusted:
                continue
            y = self.adjusted.float().cpu().numpy()
            for t in range(self.n):
                np.testing.assert_array_equal(y[t], rounded.get(t, np.full(self.V, 7.0, np.float32)), err_msg=f"row {t}")
            assert (self.out[:shift] == 7).all() and (self.out[shift + self.n * self.V:] == 7).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,shift", [(1, 0), (7, 1), (31, 0), (32, 3), (33, 0), (1000, 1), (4096, 0), (4099, 5), (20011, 0)])
def test_sizes_and_alignment(V, shift, dtype):
    _say("target", V, shift, dtype)
    s = Step(V + shift, [1, 8, 3, 64, 2], V, dtype, shift=shift, masks=0, allow=1.0)
    s.check()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("allow", [0.002, 0.5, 0.98])
@pytest.mark.parametrize("tree,lead", [(True, 1), (False, 1), (True, 0), (False, 0)])
def test_masks_trees_and_chains(tree, lead, allow, dtype):
    _say("target, masks", tree, lead, allow, dtype)
    s = Step(5, [4, 1, 17, 33, lead, 8], 3001, dtype, lead, tree=tree, allow=allow)
    want = s.want()
    s.check(status=B.STATUS_NO_TOKEN if any((y == -np.inf).all() for y in want[1].values()) else 0, want=want)


def test_a_vocabulary_in_parts():
    # few rows: each in parts, joined by a kernel of its own; one row, and rows of a large vocabulary
    _say("target, parts")
    Step(1, [1], 129280, "bf16", seen=3000, biased=300).check()
    Step(2, [2, 1], 262147, "fp32", seen=500, biased=30, masks=2, shift=1).check()


def test_many_rows_and_seen_tokens():
    # more rows than the device has workgroups, and more seen tokens than are gathered at a time
    _say("target, many")
    s = Step(3, [7] * 200, 9000, "bf16", seen=30)
    s.history.add([np.arange(0, 9000, 2).tolist()], False, [3])
    s.history.add([list(range(9000)) + [5] * 70000], True, [4])
    s.check()
    s = Step(4, [2, 1], 70000, "fp16", seen=10)
    s.history.add([list(range(70000))], False, [0])
    s.check()


@pytest.mark.parametrize("left_out", [("history",), ("drafts",), ("history", "drafts"), ("bias",), ("allowed",), ("rep", "pres"), ("rep", "freq"),
                                      ("pres", "freq"), ("rep", "pres", "freq"), ("rep", "pres", "freq", "bias", "allowed")])
def test_what_is_not_given(left_out):
    _say("target, without", left_out)
    s = Step(6, [5, 1, 9], 2003, "fp32")
    for i, name in enumerate(("rep", "pres", "freq")):
        if name in left_out:
            s.penalties[i] = None
    for name in ("history", "drafts", "bias", "allowed"):
        if name in left_out:
            setattr(s, name, None)
    want = s
    if s.history is None:
        s.history = ot.History(3, 2003)
        expect = s.want()
        s.history = None
        s.check(want=expect)
    else:
        want.check()


def test_values_that_are_not_numbers():
    _say("target, special")
    V = 5000
    for dtype in ("fp32", "bf16", "fp16"):
        s = Step(8, [8, 8, 8], V, dtype, masks=4, allow=0.5)
        s.pick = [0, 1, 2, 3, -1, 0, 1, 2] * 3 + [0] * 2
        for t in range(24):
            free = np.ones(V, bool) if s.pick[t] < 0 else s.allowed[s.pick[t]]
            on, off = np.nonzero(free)[0], np.nonzero(~free)[0]
            if t % 8 == 0:
                s.logits[t] = -math.inf                     # the lowest allowed one
            elif t % 8 == 1 and len(off):
                s.logits[t, int(off[-1])] = math.nan        # a masked one has no say
                s.logits[t, int(off[0])] = math.inf
            elif t % 8 == 2:
                s.logits[t, int(on[-1])] = s.logits[t, int(on[len(on) // 2])] = math.nan
            elif t % 8 == 3:
                s.logits[t, int(on[len(on) // 3])] = math.inf
                s.logits[t, int(on[len(on) // 2])] = math.nan
            elif t % 8 == 4:
                s.logits[t] = 0.0
                s.logits[t, 1::2] = -0.0                    # equal: the lowest one
            elif t % 8 == 5:
                s.logits[t] = -float(torch.finfo(DT[dtype]).max)
            elif t % 8 == 6:
                s.logits[t] = -math.inf
                s.logits[t, int(on[7])] = -float(torch.finfo(DT[dtype]).max)
            else:
                v = next(iter(s.history.prompt[t // 8]))    # a seen token that is not a number
                s.logits[t, v] = math.nan
                s.pick[t] = -1
        s.check()


def test_penalties_decide_near_ties_in_64_bits():
    # 5.5 / 1.1 is 5.0 in 32 bits and less in 64; it must not win over a later 5.0 there
    _say("target, near ties")
    s = Step(9, [1, 1], 100, "fp32", biased=0, masks=0, tree=False, seen=0)
    s.logits.fill_(0.0)
    s.logits[0, 3], s.logits[0, 50] = 5.5, 5.0
    s.logits[1, 3], s.logits[1, 50] = 5.0, 5.5
    for r, v in ((0, 3), (1, 50)):
        s.history.add([[v]], False, [r])
    s.penalties = [[1.1, 1.1], [0.0, 0.0], [0.0, 0.0]]
    want = s.want()
    assert want[0] == {0: 50, 1: 3}
    s.check(want=want)


def test_masks_that_allow_nothing_and_bad_rows_of_masks():
    _say("target, nothing allowed")
    s = Step(10, [3, 3], 700, "bf16", masks=3)
    s.allowed[1] = False
    s.pick = [1, 0, -1, 2, 1, 0, 0, 0]
    s.check(status=B.STATUS_NO_TOKEN)
    s.pick = [3, 0, -2, 2, 1 << 30, 0, 0, 0]
    s.check(status=B.STATUS_NO_TOKEN | B.STATUS_BAD_ROW)
    # masks of the rows themselves, further apart than they are wide
    s = Step(11, [3, 3], 700, "bf16", masks=8)
    s.pick = list(range(8))
    want = s.want()
    kw = s.prepared()
    kw["allowed"] = torch.cat((kw["allowed"], torch.full((8, 5), -1, dtype=torch.int32, device=cu.DEV)), 1)
    del kw["allowed_row"]
    s.call(kw)
    torch.cuda.synchronize()
    assert s.target.tolist() == [want[0].get(t, -7) for t in range(8)] and int(s.status.item()) == 0


def test_biases_that_do_not_fit():
    _say("target, bad biases")
    V = 900
    s = Step(12, [2, 2, 2], V, "fp32", biased=0, masks=0)
    off, val = [0, 3, 5, 9], [50.0] * 9
    for tok, mean in (([-1, 5, V, 7, 8, 1, 2, 3, 4], [[(5, 50.0)], [(7, 50.0), (8, 50.0)], [(v, 50.0) for v in (1, 2, 3, 4)]]),
                      ([1, 2, 3, 6, 6, 1, 2, 3, 4], None)):
        kw = s.prepared()
        kw["bias"] = (cu.i32(off), cu.i32(tok), torch.tensor(val, device=cu.DEV))
        s.call(kw)
        torch.cuda.synchronize()
        assert int(s.status.item()) == B.STATUS_BAD_ROW
        s.bias = mean or [[(1, 50.0), (2, 50.0), (3, 50.0)], [(6, 50.0)], [(v, 50.0) for v in (1, 2, 3, 4)]]  # one of equal entries counts
        want = s.want()
        assert s.target.tolist() == [want[0].get(t, -7) for t in range(s.n)]
    for off in ([0, 3, 2, 9], [0, 3, 5, 10], [-1, 3, 5, 9]):
        kw = s.prepared()
        kw["bias"] = (cu.i32(off), cu.i32([1, 2, 3, 7, 8, 1, 2, 3, 4]), torch.tensor(val, device=cu.DEV))
        s.call(kw)
        torch.cuda.synchronize()
        tok = [1, 2, 3, 7, 8, 1, 2, 3, 4]
        fits = [0 <= a <= b <= 9 for a, b in zip(off, off[1:])]
        if off == [0, 3, 2, 9]:
            tok[2:9] = [3, 7, 8, 1, 2, 3, 4]  # the third request's entries do not rise: of those some count
            fits[2] = None
        s.bias = [[(tok[i], 50.0) for i in range(a, b)] if f else [] for f, a, b in zip(fits, off, off[1:])]
        want = s.want()
        assert int(s.status.item()) == B.STATUS_BAD_ROW
        got = s.target.tolist()
        assert [got[t] for r in range(3) if fits[r] is not None for t in (2 * r, 2 * r + 1)] == \
            [want[0][t] for r in range(3) if fits[r] is not None for t in (2 * r, 2 * r + 1)]


def test_bad_offsets_and_drafts():
    _say("target, bad rows")
    s = Step(13, [4, 4, 4], 300, "bf16", masks=0)
    s.drafts = [-1, 300, 1 << 30, -(1 << 31)] * 3   # no tokens: they count for nothing
    s.check()
    s.drafts = [5, 6]                               # fewer than the rows have
    kw = s.prepared()
    s.call(kw)
    torch.cuda.synchronize()
    s.drafts = [5, 6] + [-1] * 20
    want = s.want()
    assert s.target.tolist() == [want[0].get(t, -7) for t in range(s.n)]
    good = Step(14, [4, 4], 300, "bf16", masks=0, tree=False)
    for offsets in ([0, 70, 6], [-1, 3, 6], [0, 3, 2_000_000_000], [0, 8, 3]):
        good.offsets = offsets
        kw = good.prepared()
        good.max_new = 4
        good.call(kw)
        torch.cuda.synchronize()
        fits = [0 <= a and 0 <= b - a + 1 <= 4 and b + r + 1 <= good.n for r, (a, b) in enumerate(zip(offsets, offsets[1:]))]
        assert int(good.status.item()) == B.STATUS_BAD_ROW and not all(fits)
        got = good.target.tolist()
        touched = {t for r, (a, b) in enumerate(zip(offsets, offsets[1:])) if fits[r] for t in range(a + r, b + r + 1)}
        assert all((got[t] != -7) == (t in touched) for t in range(good.n))


def test_strides_streams_and_captured_calls_share_a_workspace():
    _say("target, captured")
    a, b = Step(15, [3, 1], 40000, "bf16"), Step(16, [2, 8], 20001, "fp32")
    ka, kb = a.prepared(), b.prepared()
    ka["ws"] = kb["ws"] = ka["ws"] if ka["ws"].numel() > kb["ws"].numel() else kb["ws"]
    wide = torch.full((a.n, 41003), math.inf, dtype=torch.bfloat16, device=cu.DEV)   # rows of a wider tensor
    wide[:, 3:40003] = a.logits
    a.logits = wide[:, 3:40003]
    want = [s.want()[0] for s in (a, b)]
    offs = [cu.i32(s.offsets) for s in (a, b)]
    run = [lambda i=i, s=s, kw=kw: B.dspark_target_tokens(s.logits, offs[i], s.lead, s.max_new, s.target, **kw)
           for i, (s, kw) in enumerate(((a, ka), (b, kb)))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run[0]()
        run[1]()
    side.synchronize()
    for s, w in ((a, want[0]), (b, want[1])):
        assert s.target.tolist() == [w.get(t, -7) for t in range(s.n)]
    eager = [a.out.clone(), b.out.clone()]
    graphs = []
    for f in run:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for order in ((0, 1), (1, 0, 0), (1, 1, 0)):
        for s in (a, b):
            s.target.fill_(-7)
            s.out.fill_(7.0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for s, w, e in ((a, want[0], eager[0]), (b, want[1], eager[1])):
            assert s.target.tolist() == [w.get(t, -7) for t in range(s.n)] and torch.equal(s.out, e)


def test_one_workspace_for_calls_of_all_sizes():
    # rows in parts, whole rows, more rows than are counted: each call finds the counts as it needs them
    _say("target, one workspace")
    big = Step(20, [1] * 4200, 131100, "bf16", lead=1, seen=0, biased=0, masks=0, tree=False, pad=0)
    big.penalties, big.history, big.drafts = [None] * 3, None, None
    steps = [Step(21, [3, 1], 60000, "bf16"), Step(22, [1], 129280, "fp32"), Step(23, [7] * 100, 5000, "fp16"), big, Step(24, [40], 9000, "bf16")]
    ws = B.target_workspace(4200, 131100)
    want = [s.want()[0] if s is not big else None for s in steps]
    rows = big.logits.float()
    want[3] = dict(enumerate(torch.where(rows == rows.amax(1, keepdim=True), torch.arange(131100, device=cu.DEV), 131100).amin(1).tolist()))
    del rows
    for order in ((0, 1, 2, 3, 4), (4, 3, 1, 0, 2), (1, 1, 0, 3, 3)):
        for i in order:
            s = steps[i]
            kw = dict(s.prepared(adjusted=False), ws=ws)
            s.call(kw)
            torch.cuda.synchronize()
            assert s.target.tolist() == [want[i].get(t, -7) for t in range(s.n)], i
    assert not ws[:4096].any()


def test_rows_that_two_requests_have():
    # offsets that fall and rise again: those rows get one of their tokens, the others theirs, and
    # what the workspace counts does not reach the next call
    _say("target, shared rows")
    s, good = Step(25, [6, 1, 6], 60000, "bf16", lead=0, masks=0, pad=0, tree=False), Step(26, [3, 1], 60000, "bf16")
    s.penalties, s.history, s.drafts, s.bias = [None] * 3, None, None, None
    want, row = good.want()[0], s.logits.float()
    best = torch.where(row == row.amax(1, keepdim=True), torch.arange(s.V, device=cu.DEV), s.V).amin(1).tolist()
    s.offsets, ws = [0, 6, 2, 8], B.target_workspace(s.n, s.V)
    ws[4096:] = -1
    for _ in range(40):
        kw = dict(s.prepared(adjusted=False), ws=ws)
        s.call(kw)
        torch.cuda.synchronize()
        got = s.target.tolist()
        assert int(s.status.item()) & B.STATUS_BAD_ROW
        assert got[:2] + got[6:] == best[:2] + best[6:8] + [-7] * 5
        assert all(0 <= v < s.V for v in got[2:6])
        assert not ws[:4096].any()
        good.call(dict(good.prepared(adjusted=False), ws=ws))
        torch.cuda.synchronize()
        assert good.target.tolist() == [want.get(t, -7) for t in range(good.n)]


@pytest.mark.parametrize("penalty", [(0.25, 0.0, 0.0), (1.0, -3.0, 0.0), (1.0, 0.0, -0.5), (0.8, -0.5, 0.0), (0.9, 0.25, -0.25), (0.0, 0.0, 0.0),
                                     (-1.5, 0.0, 0.0), (1e-30, 0.0, 0.0), (1e30, 0.0, 0.0), (1.2, math.inf, 0.0), (1.0, -math.inf, 0.0),
                                     (math.inf, 0.0, 0.0), (math.nan, 0.0, 0.0), (1.0, math.nan, 0.0)])
def test_penalties_that_lift_or_are_no_numbers(penalty):
    # tokens whose logits alone would never win, and every value that a parameter may have
    _say("target, lifting penalties", penalty)
    for dtype, V in (("fp32", 5003), ("bf16", 9000)):
        s = Step(30, [5, 1, 12], V, dtype, seen=60, biased=4)
        s.logits -= 6.0 if penalty[0] < 1 else 0.0  # negative ones are lifted by a repetition below one
        s.penalties = [[p] * 3 for p in penalty]
        s.check()


@pytest.mark.parametrize("rows,V,n,width", [(1, 1, 1, 5), (4, 130, 3, 70), (9, 4096, 9, 1), (5, 70001, 40, 3000), (2, 600001, 3, 700),
                                               (3, 1001, 4, 40000), (2, 524288, 2, 256), (2, 262144, 2, 9000), (2, 7, 2, 20000)])
def test_history(rows, V, n, width):
    _say("history", rows, V, n, width)
    rng = np.random.default_rng(V)
    h, w, status = B.History(rows, V, device=cu.DEV), ot.History(rows, V), torch.zeros(1, dtype=torch.int32, device=cu.DEV)

    def same(bits):
        torch.cuda.synchronize()
        seen, count = w.arrays()
        np.testing.assert_array_equal(h.seen.cpu().numpy(), seen)
        np.testing.assert_array_equal(h.count.cpu().numpy(), count)
        assert int(status.item()) == bits
    for answered in (False, True, True):
        tokens = (rng.random((n, width)) ** 3 * (V + 1)).astype(int) - (rng.random((n, width)) < 0.2)
        tokens = np.minimum(tokens, V - 1)
        to = rng.integers(0, rows, n).tolist()      # a row more than once
        w.add(tokens.tolist(), answered, to)
        B.dspark_history_add(h, cu.i32(tokens), answered, rows=cu.i32(to), status=status)
        same(0)
    B.dspark_history_clear(h, cu.i32([rows - 1] * 3), status=status)
    w.clear([rows - 1])
    same(0)
    assert w.add([[V, 0], [1 << 30, -5]][:1], True, [0]) == w.add([[0]], False, [rows]) == w.clear([-1]) == ot.BAD_ROW
    B.dspark_history_add(h, cu.i32([[V, 0]]), True, rows=cu.i32([0]), status=status)
    B.dspark_history_add(h, cu.i32([[0]]), False, rows=cu.i32([rows]), status=status)
    B.dspark_history_clear(h, cu.i32([-1]), status=status)
    same(B.STATUS_BAD_ROW)
    B.dspark_history_clear(h)
    torch.cuda.synchronize()
    assert not h.seen.any() and not h.count.any()


def test_history_past_32_bits():
    # counts numbered past 2^32
    _say("history, large")
    rows, V = 4500, 1 << 20
    h = B.History(rows, V, device=cu.DEV)
    B.dspark_history_add(h, cu.i32([[5, 5, V - 1]]), True, rows=cu.i32([rows - 1]))
    torch.cuda.synchronize()
    assert h.count[-1, 5] == 2 and h.count[-1, V - 1] == 1
    assert int(h.count.sum()) == 3
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device=cu.DEV)
    x[-1, 5], x[-1, V - 1], x[-1, 9] = 3.0, 2.0, 1.5
    target = torch.full((rows,), -7, dtype=torch.int32, device=cu.DEV)
    f = torch.full((rows,), 0.5, device=cu.DEV)
    B.dspark_target_tokens(x, cu.i32(np.zeros(rows + 1)), 1, 1, target, history=h, penalties=(None, None, f * 2), ws=B.target_workspace(rows, V))
    torch.cuda.synchronize()
    assert target[-1].item() == 9 and (target[:-1] == 0).all()  # 3 - 2, 2 - 1 and 1.5
    B.dspark_history_clear(h, cu.i32([rows - 1]))
    torch.cuda.synchronize()
    assert not h.seen.any() and int(h.count.sum()) == 0


def test_history_of_the_widest_rows():
    # entry numbers up to the last one that 32 bits hold (8 GiB of tokens)
    _say("history, widest rows")
    width = (1 << 31) - 1
    tokens = torch.full((1, width), -1, dtype=torch.int32, device=cu.DEV)
    for at, v in ((0, 3), (width // 2, 3), (width - 65536, 4), (width - 1, 5)):
        tokens[0, at] = v
    h, status = B.History(2, 40, device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    B.dspark_history_add(h, tokens, True, rows=cu.i32([1]), status=status)
    B.dspark_history_add(h, tokens, False, rows=cu.i32([0]), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert h.count[1].tolist() == [0, 0, 0, 2, 1, 1] + [0] * 34 and not h.count[0].any()
    assert h.seen[:, :, 0].tolist() == [[0b111000, 0], [0, 0b111000]] and not h.seen[:, :, 1:].any()


@pytest.mark.parametrize("frequency", [math.inf, -math.inf, math.nan])
def test_frequencies_that_are_no_numbers_reach_what_was_answered_alone(frequency):
    # not the prompt's tokens, nor those that only a bias changes
    _say("target, frequency", frequency)
    for dtype, V, seen in (("fp32", 5003, 0), ("bf16", 9000, 1), ("bf16", 5003, 60)):
        s = Step(40, [5, 1, 12], V, dtype, seen=seen, biased=6)
        s.penalties = [[1.0] * 3, [0.25] * 3, [frequency] * 3]
        if seen < 2:  # and nothing has been answered
            s.drafts = None
        s.check()


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3.4e38, -3.4e38])
def test_biases_of_any_value(value):
    _say("target, biases", value)
    for dtype, V in (("fp32", 5003), ("fp16", 9000)):
        s = Step(41, [5, 1, 12], V, dtype, biased=6)
        s.bias = [[(v, value if i % 2 else b) for i, (v, b) in enumerate(x)] for x in s.bias]
        s.check()


@pytest.mark.parametrize("V,rows,dtype", [(700, [3, 3, 2], "bf16"), (40000, [2, 1], "fp32"), (9000, [64] * 8, "fp16")])
def test_rows_without_a_token_can_have_none(V, rows, dtype):
    # whole rows, rows in parts, many rows
    _say("target, none", V, len(rows), dtype)
    s = Step(50, rows, V, dtype, masks=3, biased=0, seen=3, tree=False)
    s.allowed[1] = False
    s.pick = [(1, 0, 2, -1, 3)[t * 7 % 5] for t in range(s.n)]
    for token in (-1, 0, 5, V - 1):
        kw = s.prepared(adjusted=False)
        s.call(dict(kw, no_token=token))
        torch.cuda.synchronize()
        if token == -1:
            want = s.want()[0]
            empty = {t for t in want if s.pick[t] in (1, 3)}
            assert empty and len(empty) < len(want)
        assert s.target.tolist() == [token if t in empty else want.get(t, -7) for t in range(s.n)]
        assert int(s.status.item()) == B.STATUS_NO_TOKEN | B.STATUS_BAD_ROW


def test_a_draft_does_not_pass_a_mask_that_allows_nothing():
    # a path ends at a row without a token, whose answer is none: for trees, chains and the history
    _say("target, none accepted")
    V, off = 50, cu.i32([0, 3])
    x = torch.zeros((4, V), device=cu.DEV)
    x[0, 4], x[1, 0], x[2, 0], x[3, 9] = 1.0, 1.0, 1.0, 1.0   # the drafts 4, 0, 0 and then 9 without masks
    drafts, parent = cu.i32([4, 0, 0]), cu.i32([-1, 0, 1, 2])
    allowed = _pack(np.stack([np.ones(V, bool), np.zeros(V, bool)]))
    new = lambda *n: torch.full(n, 7, dtype=torch.int32, device=cu.DEV)  # noqa: E731
    for token, out in ((0, [4, 0, 0, 9]), (-1, [4, -1, -1, -1])):
        target, status = new(4), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
        B.dspark_target_tokens(x, off, 1, 4, target, allowed=allowed, allowed_row=cu.i32([0, 1, 0, 0]), status=status, no_token=token,
                               ws=B.target_workspace(4, V))
        accept, path, bonus, answer = new(1), new(1, 3), new(1), new(1, 4)
        B.dspark_accept_tree(drafts, off, parent, target, accept, path, bonus, out_tokens=answer, status=status)
        h = B.History(1, V, device=cu.DEV)
        B.dspark_history_add(h, answer, True, status=status)
        torch.cuda.synchronize()
        assert target.tolist() == [4, token, 0, 9] and int(status.item()) == B.STATUS_NO_TOKEN
        assert answer.tolist() == [out] and accept.item() == sum(v >= 0 for v in out) - (token == 0) and bonus.item() == (9 if token == 0 else -1)
        counts = [0] * V
        for v in out:
            if v >= 0:
                counts[v] += 1
        assert h.count[0].tolist() == counts


def test_more_rows_than_are_counted_can_have_none():
    # their parts are joined by a kernel of its own
    _say("target, none of many")
    n, V = 4100, 131100
    x = torch.zeros((n, V), dtype=torch.bfloat16, device=cu.DEV)
    x[:, V - 1] = 1.0
    pick = np.arange(n) % 3 - 1
    target, status = torch.full((n,), -7, dtype=torch.int32, device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    allowed = _pack(np.stack([np.arange(V) < V - 1, np.zeros(V, bool)]))
    for token in (-1, 0):
        B.dspark_target_tokens(x, cu.i32(np.zeros(n + 1)), 1, 1, target, allowed=allowed, allowed_row=cu.i32(pick), status=status,
                               no_token=token, ws=B.target_workspace(n, V))
        torch.cuda.synchronize()
        assert target.tolist() == [(V - 1, 0, token)[p + 1] for p in pick.tolist()] and int(status.item()) == B.STATUS_NO_TOKEN


@pytest.mark.parametrize("V,rows", [(5003, [2, 1, 3, 1]), (40001, [1, 1, 1, 1]), (9000, [8] * 4)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_biases(V, rows, dtype):
    # as many as stand in LDS, one fewer and more; in whole rows and in parts
    _say("target, many biases", V, rows, dtype)
    for masks in (0, 2):
        s = Step(60, rows, V, dtype, masks=masks)
        s.bias = [[(int(v), float(np.float32(s.rng.standard_normal()))) for v in np.sort(s.rng.choice(V, n, replace=False))]
                  for n in (511, 512, 513, 2000)]
        s.check()


def test_a_late_bias_that_does_not_rise():
    # beyond those that stand in LDS: reported; other requests are served
    _say("target, late bias")
    V = 3001
    s = Step(61, [2, 3], V, "fp32", masks=0)
    tok = list(range(0, 1400, 2))
    s.bias = [[(v, 0.25) for v in tok], [(3, 1.0), (9, 2.0)]]
    want = s.want()[0]
    kw = s.prepared(adjusted=False)
    for at, v in ((699, 1396), (600, 5), (513, -1), (512, V), (699, 1 << 30)):
        bad = list(tok)
        bad[at] = v
        s.status.zero_()
        kw["bias"] = (cu.i32([0, 700, 702]), cu.i32(bad + [3, 9]), torch.tensor([0.25] * 700 + [1.0, 2.0], device=cu.DEV))
        s.call(kw)
        torch.cuda.synchronize()
        assert int(s.status.item()) == B.STATUS_BAD_ROW, (at, v)
        got = s.target.tolist()
        assert got[2:5] == [want[t] for t in (2, 3, 4)] and all(0 <= x < V for x in got[:2]) and got[5:] == [-7] * (s.n - 5)


@pytest.mark.parametrize("lead", [0, 1])
@pytest.mark.parametrize("V,rows,dtype", [(3001, [256, 65, 1], "bf16"), (2003, [200, 64, 128], "fp32"), (40001, [100, 1, 66], "fp16")])
def test_long_chains(V, rows, dtype, lead):
    # up to 256 rows of a request, each with the drafts before it, many of them more than once
    _say("target, long chains", V, rows, dtype, lead)
    s = Step(62, rows, V, dtype, lead, tree=False, masks=2, biased=20)
    s.drafts = [int(v) for v in s.rng.choice(s.rng.choice(V, 40, replace=False), s.n)]
    s.check()
    s.penalties = [[0.8, 1.2, 1.0], [-0.5, 0.25, 0.0], [0.05, -0.05, 0.5]]
    s.check()


def test_the_largest_vocabulary():
    _say("target, 2^30 tokens")
    V = 1 << 30
    x = torch.zeros((1, V), dtype=torch.bfloat16, device=cu.DEV)
    at = [5, 131072 * 4000 + 17, V - 131072, V - 9, V - 1]
    x[0, at] = torch.tensor([1.0, 3.0, 2.0, 4.0, 5.0], dtype=torch.bfloat16, device=cu.DEV)
    h, status = B.History(1, V, device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    B.dspark_history_add(h, cu.i32([[V - 1, V - 1, V - 9, V]]), True, status=status)
    B.dspark_history_add(h, cu.i32([[5] * 300]), False, status=status)
    target, out = torch.full((1,), -7, dtype=torch.int32, device=cu.DEV), torch.full_like(x, 7.0)
    one = lambda v: torch.full((1,), v, device=cu.DEV)  # noqa: E731
    ws = B.target_workspace(1, V)
    for adjusted in (None, out):
        target.fill_(-7)
        B.dspark_target_tokens(x, cu.i32([0, 0]), 1, 1, target, history=h, penalties=(one(2.0), one(0.25), one(0.5)), adjusted=adjusted, ws=ws,
                               bias=(cu.i32([0, 2]), cu.i32([7, V - 131072]), torch.tensor([2.9, 1.5], device=cu.DEV)), status=status)
        torch.cuda.synchronize()
        assert target.item() == V - 131072 and int(status.item()) == B.STATUS_BAD_ROW  # 3.5, of 0.5, 3.0, 3.5, 1.25 and 1.25
    assert out[0, at].tolist() == [0.5, 3.0, 3.5, 1.25, 1.25] and abs(out[0, 7].item() - 2.9) <= 2.9 * 2.0 ** -8
    out[0, at + [7]] = 0
    assert not out.any()


def test_the_most_rows():
    # as many requests as there may be, of as many rows, each with the drafts before it
    _say("target, 8192 requests of 256 rows")
    R, n, V = 8192, 256, 11
    g = torch.Generator(device=cu.DEV).manual_seed(1)
    x = torch.randint(0, 9, (R * n, V), generator=g, device=cu.DEV).to(torch.float16)
    drafts = torch.randint(0, V, (R, n), generator=g, device=cu.DEV, dtype=torch.int32)
    target = torch.full((R * n,), -7, dtype=torch.int32, device=cu.DEV)
    off = (torch.arange(R + 1, device=cu.DEV) * n).int()
    B.dspark_target_tokens(x, off, 0, n, target, penalties=(None, None, torch.full((R,), 0.25, device=cu.DEV)), node_tokens=drafts.view(-1),
                           ws=B.target_workspace(R * n, V))
    said = torch.nn.functional.one_hot(drafts.long(), V).cumsum(1).view(R * n, V)
    want = x.float() - 0.25 * said  # exact
    best = torch.where(want == want.amax(1, keepdim=True), torch.arange(V, device=cu.DEV), V).amin(1)
    torch.cuda.synchronize()
    assert torch.equal(target, best.int())


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_processed_rows_of_a_wider_tensor(dtype):
    _say("target, wide adjusted", dtype)
    for V, gap, first in ((3001, 5, 3), (40000, 7, 1), (64, 1, 0)):
        s = Step(70, [3, 1, 6], V, dtype)
        want = s.want()
        kw = s.prepared(adjusted=False)
        wide = torch.full((s.n, V + gap), 7.0, dtype=DT[dtype], device=cu.DEV)
        kw["adjusted"] = wide[:, first:first + V]
        s.call(kw)
        torch.cuda.synchronize()
        assert s.target.tolist() == [want[0].get(t, -7) for t in range(s.n)]
        for t in range(s.n):
            y = np.full(V + gap, 7.0, np.float32)
            if t in want[1]:
                y[first:first + V] = torch.from_numpy(want[1][t]).float().to(DT[dtype]).float().numpy()
            np.testing.assert_array_equal(wide[t].float().cpu().numpy(), y)


def test_two_calls_at_once():
    # on two streams, with a workspace each: one history and one set of logits read by both
    _say("target, two streams")
    s = Step(71, [3, 1, 6], 60000, "bf16")
    want = [s.want()[0].get(t, -7) for t in range(s.n)]
    kw, off = s.prepared(adjusted=False), cu.i32(s.offsets)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.full_like(s.target, -7) for _ in streams]
    ws = [B.target_workspace(s.n, s.V) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(50):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].fill_(-7)
                B.dspark_target_tokens(s.logits, off, s.lead, s.max_new, got[i], **dict(kw, ws=ws[i]))
    torch.cuda.synchronize()
    assert [x.tolist() for x in got] == [want, want]
