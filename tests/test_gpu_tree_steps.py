"""Verification steps of drafted trees as an engine runs them: chains sampled under several
seeds and scheduled, merged into trees, planned, pages reserved, keys and queries turned
and appended, attention, the target's choice under penalties and masks, acceptance, the
path's K and V moved, commit, history -- every buffer against the oracle, alone and as one
captured graph."""
import math

import numpy as np
import pytest
import torch

import cache_util as cu
import gpu_util as gu
from confidence_scheduled_verification_amd import binding as B
from confidence_scheduled_verification_amd import inputs
from oracle import cache as oc
from oracle import tree as ot
from test_gpu_tree import signed

pytestmark = pytest.mark.gpu

R, S, K, V, H, HKV, D, PAGE, LAYERS = 6, 4, 5, 1024, 4, 2, 64, 16, 2
N = R * (S * K + 1)  # rows of a step at most


def _say(*a):
    print(*a, flush=True)


def _i(*shape, value=0):
    return torch.full(shape, value, dtype=torch.int32, device=cu.DEV)


class Engine:
    def __init__(self, seed):
        self.rng = rng = np.random.default_rng(seed)
        width, n_pages = 14, 90
        self.st = st = cu.State(rng, LAYERS, n_pages, PAGE, HKV, D, "bf16", R, width, fill=0.0)
        self.prefix = [40, 7]                      # two pages that all requests begin with
        for p in self.prefix:
            st.ref[p] = R - 1
        for la in range(LAYERS):
            st.put(la, self.prefix, 0, 2 * PAGE)
        for r in range(R):
            st.table[r][:2], st.len[r] = self.prefix, 2 * PAGE
        st.table[2], st.len[2] = [-1] * width, -1   # a slot without a request
        self.cache = st.upload()
        case = inputs.random_case(seed, R=R * S, K=K, V=V, rank=32, dtype=inputs.BF16, base_std=1.0)
        base = np.repeat(case["base"][::S], S, 0)   # a request's chains come from the same logits
        self.chain = gu.Chain(base, case["A"], case["Bmat"], inputs.BF16, case["prev0"])
        w = inputs.WORKLOADS["small"]
        self.vc = torch.from_numpy(B.dspark_force_monotone(inputs.raw_verify_cost(w, None))).to(cu.DEV)
        self.dc = torch.from_numpy(B.dspark_force_monotone(inputs.raw_draft_cost(w))).to(cu.DEV)
        self.history, self.said = B.History(R, V, device=cu.DEV), ot.History(R, V)
        prompt = rng.integers(0, V, (R, 40))
        B.dspark_history_add(self.history, cu.i32(prompt), answered=False)
        self.said.add(prompt.tolist(), False, range(R))
        self.rotary = B.Rotary(64, 10000.0, scaling="linear", factor=2.0)
        self.pen = [np.float32(rng.uniform(a, b, R)) for a, b in ((1.0, 1.4), (0.0, 0.5), (0.0, 0.3))]
        self.d_pen = tuple(torch.from_numpy(x).to(cu.DEV) for x in self.pen)
        self.ws, self.page_ws = B.cache_workspace(self.cache, R, H, S * K + 1, 1), B.pages_workspace(self.cache, R)
        self.t_ws = B.target_workspace(N, V)
        self.shared = (cu.i32([0, R]), cu.i32([self.prefix]), cu.i32([2]))
        self.out = B.StepBuffers(R * S, K)
        names = dict(tokens=(R * S, K), counts=(R,), offsets=(R + 1,), drafts=(R * S * K,), parent=(N,), depth=(N,), granted=(R,),
                     target=(N,), accept=(R,), path=(R, K), nxt=(R,), emitted=(R, K + 1), status=(1,))
        self.b = {k: _i(*shape) for k, shape in names.items()}
        self.anc = torch.zeros(N, dtype=torch.int64, device=cu.DEV)
        self.q_out, self.res = (torch.zeros((LAYERS, N, H, D), dtype=torch.bfloat16, device=cu.DEV) for _ in range(2))
        self.lse = torch.zeros((LAYERS, N, H), device=cu.DEV)
        self.prev = _i(R * S)

    def inputs(self):
        """What changes from step to step: confidences, the model's q, k, v and logits, the grammar's masks."""
        rng = self.rng
        qkv = torch.randn((LAYERS, N, H + 2 * HKV, D), device=cu.DEV).bfloat16()
        logits = cu.rounded(rng.standard_normal((N, V)), "bf16").to(cu.DEV)
        allowed = torch.from_numpy(rng.integers(-(1 << 31), 1 << 31, (3, V // 32)).astype(np.int32)).to(cu.DEV)
        conf = torch.from_numpy(rng.uniform(0.5, 1.0, (R * S, K)).astype(np.float32)).to(cu.DEV)
        return dict(qkv=qkv, logits=logits, allowed=allowed, pick=cu.i32(rng.integers(-1, 3, N)), conf=conf)

    def before_target(self, x):
        b, c = self.b, self.cache
        B.dspark_chain_sample(self.chain.base, self.chain.markov, self.prev, 1.0, 7, b["tokens"], None, b["status"], self.chain.ws)
        B.dspark_schedule(x["conf"], R, 0, R, self.vc, self.dc, self.out, tokens=b["tokens"], status=b["status"])
        B.dspark_tree_merge(b["tokens"], self.out.prefix_len, S, b["counts"], b["offsets"], b["drafts"], b["parent"], b["status"])
        B.dspark_tree_plan(b["parent"], b["offsets"], 1, S * K + 1, b["depth"], self.anc, b["status"])
        B.dspark_pages_reserve(c, b["offsets"], 1, b["granted"], self.page_ws, b["status"])
        for la in range(LAYERS):
            q, k, v = (x["qkv"][la, :, i:j] for i, j in ((0, H), (H, H + HKV), (H + HKV, H + 2 * HKV)))
            B.dspark_cache_append_rotary(c, la, self.rotary, q, self.q_out[la], k, v, b["offsets"], 1, S * K + 1, depth=b["depth"],
                                         status=b["status"])
            B.dspark_cache_attend_tree(c, la, self.q_out[la], b["offsets"], 1, S * K + 1, self.anc, 0.125, self.res[la],
                                       lse=self.lse[la], shared=self.shared, ws=self.ws, status=b["status"])

    def choose(self, x):
        b = self.b
        B.dspark_target_tokens(x["logits"], b["offsets"], 1, S * K + 1, b["target"], history=self.history, penalties=self.d_pen,
                               node_tokens=b["drafts"], anc=self.anc, allowed=x["allowed"], allowed_row=x["pick"], ws=self.t_ws,
                               status=b["status"])

    def after_target(self):
        b, c = self.b, self.cache
        B.dspark_accept_tree(b["drafts"], b["offsets"], b["parent"], b["target"], b["accept"], b["path"], b["nxt"], b["emitted"],
                             b["status"])
        B.dspark_cache_keep_path(c, b["path"], b["accept"], 1, granted=b["granted"], status=b["status"])
        B.dspark_pages_commit(c, b["accept"], 1, status=b["status"], granted=b["granted"])
        B.dspark_history_add(self.history, b["emitted"], answered=True, status=b["status"])

    def lean(self, x):
        """Logits that agree with the drafts along one chain of each request, so that paths are accepted."""
        torch.cuda.synchronize()
        b = {k: t.tolist() for k, t in self.b.items()}
        anc = self.anc.tolist()
        for r in range(R):
            row, n = b["offsets"][r] + r, b["counts"][r]
            if not n:
                continue
            last = int(self.rng.integers(1, n + 1))
            way = [j for j in range(n + 1) if anc[row + last] >> j & 1]
            for at, j in zip(way, way[1:]):
                x["logits"][row + at, b["drafts"][b["offsets"][r] + j - 1]] = 30.0
                x["pick"][row + at] = -1


def test_tree_steps():
    e = Engine(21)
    st, kept = e.st, 0
    for step in range(5):
        _say("tree step", step)
        x = e.inputs()
        e.before_target(x)
        e.lean(x)
        e.choose(x)
        e.after_target()
        torch.cuda.synchronize()
        b = {k: t.tolist() for k, t in e.b.items()}
        # the tree
        lens = e.out.prefix_len.view(R, S).tolist()
        counts, offsets, drafts, parent, bad = ot.merge(e.b["tokens"].view(R, S, K).tolist(), lens)
        n, depth, anc = len(parent), [0] * len(parent), [0] * len(parent)
        bad |= ot.plan(parent, offsets, 1, 64, depth, anc)
        assert (b["counts"], b["offsets"], b["drafts"][:len(drafts)], b["parent"][:n]) == (counts, offsets, drafts, parent)
        assert b["depth"][:n] == depth and e.anc.tolist()[:n] == signed(anc)
        # the cache and attention, layer by layer, from the K that the kernel wrote (its rounding is its own)
        granted, s = oc.reserve(st.table, st.len, st.ref, offsets, 1, PAGE)
        assert b["granted"] == granted
        bad |= s
        for la in range(LAYERS):
            qkv = x["qkv"][la].cpu().double().numpy()
            for r in range(R):
                a0, b0 = oc.rows_of(offsets, 1, r)
                if st.len[r] < 0:
                    continue
                pos = [st.len[r] + depth[t] for t in range(a0, b0)]
                turned, reach = ot.rotate(qkv[a0:b0, :H + HKV], pos, e.rotary.freq, 64, 0, False, 1.0)
                near = 2.0 ** -21 * reach + 2.0 ** -8 * np.abs(turned) + 2.0 ** -25  # see test_gpu_rotary
                q = e.q_out[la, a0:b0].cpu().double().numpy()
                assert (np.abs(q - turned[:, :H]) <= near[:, :H]).all()
                k = cu.rounded(turned[:, H:], "bf16").double().numpy()  # the nearest 16-bit values, or their neighbours
                for i in range(b0 - a0):
                    p = st.len[r] + i
                    st.k[la, st.table[r][p // PAGE], :, p % PAGE] = k[i]
                    st.v[la, st.table[r][p // PAGE], :, p % PAGE] = qkv[a0 + i, H + HKV:]
        # target, acceptance, path, commit
        target = []
        for r in range(R):
            a0, b0 = oc.rows_of(offsets, 1, r)
            for t in range(a0, b0):
                path = [drafts[offsets[r] + i - 1] for i in range(1, b0 - a0) if anc[t] >> i & 1]
                pick = int(x["pick"][t])
                free = None if pick < 0 else np.unpackbits(x["allowed"][pick].cpu().numpy().view(np.uint8), bitorder="little").astype(bool)
                target.append(ot.choose(x["logits"][t].double().cpu().numpy(), path, e.said.prompt[r], e.said.count[r],
                                        *(float(p[r]) for p in e.pen), None, free)[0])
        assert b["target"][:n] == target
        accept, path, nxt, emitted, s = ot.accept(drafts, offsets, parent, target, K)
        bad |= s
        assert (b["accept"], b["path"], b["nxt"], b["emitted"]) == (accept, path, nxt, emitted)
        kept += sum(accept)
        # attention read the cache as it stood before the path was moved
        moved_k, moved_v = st.k.copy(), st.v.copy()
        bad |= ot.keep_path(moved_k, moved_v, st.table, st.len, st.ref, path, accept, 1, granted)
        for la in range(LAYERS):
            want = ot.attend(e.q_out[la, :n].cpu().double().numpy(), st.k[la], st.v[la], st.table, st.len, offsets, 1, 0.125, anc)
            # K may stand one rounding beside the kernel's: 2^-8 of it, and so of a score's reach
            out, lse, spread, reach = want
            off = 2.0 ** -7 * reach
            got, glse = e.res[la, :n].cpu().double().numpy(), e.lse[la, :n].cpu().double().numpy()
            b_out, b_lse = cu.attend_bounds(want, "bf16", 300, D)
            seen = np.isfinite(lse)
            assert (np.abs(got - out)[seen] <= (b_out + (2 * off[..., None]) * spread * 1.2)[seen]).all()
            assert (np.abs(glse[seen] - lse[seen]) <= (b_lse + off)[seen]).all() and (got[~seen] == 0).all()
        st.k[:], st.v[:] = moved_k, moved_v
        bad |= oc.commit(st.table, st.len, st.ref, accept, 1, PAGE, granted)
        e.said.add(emitted, True, range(R))
        assert int(e.b["status"].item()) == bad
        e.b["status"].zero_()
        st.assert_books()
        # K to a rounding (then the kernel's), V bit for bit, wherever a row's tokens stand
        k, v = oc.unpack_k(e.cache.k.cpu().double().numpy()), oc.unpack_v(e.cache.v.cpu().double().numpy())
        for r in range(R):
            for p in range(max(st.len[r], 0)):
                at = (slice(None), st.table[r][p // PAGE], slice(None), p % PAGE)
                np.testing.assert_array_equal(v[at], st.v[at])
                assert (np.abs(k[at] - st.k[at]) <= 2.0 ** -7 * np.abs(st.k[at]) + 2.0 ** -16).all(), (r, p)
        st.k[:] = k
        st.v[:] = v
        seen, count = e.said.arrays()
        np.testing.assert_array_equal(e.history.seen.cpu().numpy(), seen)
        np.testing.assert_array_equal(e.history.count.cpu().numpy(), count)
    assert kept >= 10


def test_a_captured_step():
    # the whole step as one graph, replayed from the same state: every replay gives what the calls gave
    _say("tree step, captured")
    e = Engine(22)
    x = e.inputs()
    state = dict(k=e.cache.k, v=e.cache.v, table=e.cache.table, len=e.cache.len, ref=e.cache.ref, seen=e.history.seen, count=e.history.count)
    start = {k: t.clone() for k, t in state.items()}
    made = dict(e.b, anc=e.anc, res=e.res, lse=e.lse, q=e.q_out, **state)

    def again():
        for k, t in start.items():
            state[k].copy_(t)
        for k, t in made.items():
            if k not in state:
                t.zero_()

    def step():
        e.before_target(x)
        e.choose(x)
        e.after_target()
    e.before_target(x)
    e.lean(x)
    again()
    step()
    torch.cuda.synchronize()
    want = {k: t.clone() for k, t in made.items()}
    assert int(want["accept"].sum()) > 0 and int(want["status"].item()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        again()
        e.ws.fill_(0x7FC00000)
        e.t_ws[4096:] = -1
        graph.replay()
        torch.cuda.synchronize()
        for k, t in made.items():
            assert torch.equal(t, want[k]), k
    assert math.isfinite(float(want["res"].float().sum()))
