"""CPU checks of the trees', rotary and target entry points: what they refuse before any HIP
call, what the binding refuses, and the host-side frequencies.  No kernel runs."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from confidence_scheduled_verification_amd import binding as B
from oracle import tree as ot
from test_cache_host import DATA, _cache, _fake

KEEP = []


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_merge_plan_and_accept_refuse():
    L, p = B.lib(), _fake()

    def merge(t=p, ln=p, R=2, S=3, K=4, c=p, o=p, v=p, par=p):
        return L.dspark_tree_merge(t, ln, R, S, K, c, o, v, par, None, None)
    for kw, rc in ((dict(R=-1), -2), (dict(S=0), -2), (dict(K=0), -2), (dict(S=8, K=8), -3), (dict(S=1 << 20, K=1 << 20), -3),
                   (dict(R=8193), -3), (dict(t=None), -1), (dict(c=None), -1), (dict(o=None), -1), (dict(v=None), -1),
                   (dict(par=None), -1)):
        assert merge(**kw) == rc, kw
    assert merge(t=None, R=0) == 0 and L.dspark_last_error()

    def plan(par=p, n=10, o=p, lead=1, R=2, most=8, d=p, a=p):
        return L.dspark_tree_plan(par, n, o, lead, R, most, d, a, None, None)
    for kw, rc in ((dict(n=-1), -2), (dict(lead=2), -2), (dict(R=-1), -2), (dict(R=8193), -3), (dict(most=-1), -2), (dict(most=65), -3),
                   (dict(par=None), -1), (dict(o=None), -1), (dict(d=None), -1), (dict(a=None), -1)):
        assert plan(**kw) == rc, kw
    for kw in (dict(R=0), dict(n=0), dict(most=0)):
        assert plan(par=None, o=None, d=None, a=None, **kw) == 0

    def accept(v=p, n=10, o=p, par=p, t=p, R=2, K=4, al=p, path=p, nx=p):
        return L.dspark_accept_tree(v, n, o, par, t, R, K, al, path, nx, None, None, None)
    for kw, rc in ((dict(n=-1), -2), (dict(R=-1), -2), (dict(K=-1), -2), (dict(K=64), -2), (dict(n=(1 << 31) - 1), -3), (dict(v=None), -1),
                   (dict(o=None), -1), (dict(par=None), -1), (dict(t=None), -1), (dict(al=None), -1), (dict(path=None), -1),
                   (dict(nx=None), -1)):
        assert accept(**kw) == rc, kw
    assert accept(v=None, o=None, par=None, t=None, al=None, path=None, nx=None, R=0) == 0


def test_keep_path_refuses():
    L, p = B.lib(), _fake()

    def call(c=None, path=p, K=4, a=p, lead=1, R=4):
        return L.dspark_cache_keep_path(c or _cache(), path, K, a, None, lead, R, None, None)
    for kw, rc in DATA:
        assert call(_cache(**kw)) == rc, kw
    for kw, rc in ((dict(path=None), -1), (dict(a=None), -1), (dict(K=-1), -2), (dict(K=64), -2), (dict(lead=2), -2), (dict(R=9), -2),
                   (dict(R=-1), -2), (dict(c=_cache(layers=1 << 17)), -3)):
        assert call(**kw) == rc, kw
    assert call(path=None, a=None, R=0) == 0


def test_attend_tree_refuses():
    L, p, ws = B.lib(), _fake(), _fake(4096)

    def call(c=None, layer=0, q=p, qs=256, rows=4, H=4, off=p, lead=1, R=4, most=8, anc=p, scale=0.125, ng=0, ws=ws, n=1 << 40):
        return L.dspark_cache_attend_tree(c or _cache(), layer, q, qs, rows, H, off, lead, R, most, anc, scale, ng, None, None, 0,
                                          None, p, 256, None, None, ws, n, None)
    for kw, rc in DATA:
        assert call(_cache(**kw)) == rc, kw
    for kw, rc in ((dict(most=65), -3), (dict(anc=None), -1), (dict(layer=2), -2), (dict(q=None), -1), (dict(H=3), -1), (dict(off=None), -1),
                   (dict(scale=0.0), -2), (dict(ng=1), -1), (dict(ws=None), -4), (dict(ws=ws + 8), -1)):
        assert call(**kw) == rc, kw
    for kw in (dict(R=0), dict(rows=0), dict(most=0)):
        assert call(q=None, off=None, anc=None, ws=None, **kw) == 0


def _rotary(**kw):
    f = dict(turns=_fake(), dim=32, first=0, interleaved=0, attention=1.0)
    f.update(kw)
    r = B.dspark_rotary_t(*[f[n] for n, _ in B.dspark_rotary_t._fields_])
    KEEP.append(r)
    return ctypes.byref(r)


def test_append_rotary_refuses():
    L, p, far = B.lib(), _fake(), _fake(1 << 14)

    def call(c=None, layer=0, rot=None, q=p, qs=256, H=4, out=far, os_=256, k=p, ks=128, v=p, vs=128, rows=4, off=p, lead=1, R=4, most=8):
        return L.dspark_cache_append_rotary(c or _cache(), layer, rot or _rotary(), q, qs, H, out, os_, k, ks, v, vs, rows, off, lead,
                                            R, most, None, None, None)
    for kw, rc in DATA:
        assert call(_cache(**kw)) == rc, kw
    for kw, rc in ((dict(dim=0), -1), (dict(dim=8), -1), (dict(dim=24), -1), (dict(dim=80), -1), (dict(first=4), -1), (dict(first=-8), -1),
                   (dict(first=40), -1), (dict(attention=math.nan), -2), (dict(attention=math.inf), -2), (dict(turns=None), -1)):
        assert call(rot=_rotary(**kw)) == rc, kw
    assert L.dspark_cache_append_rotary(_cache(), 0, None, p, 256, 4, far, 256, p, 128, p, 128, 4, p, 1, 4, 8, None, None, None) == -1
    for kw, rc in ((dict(layer=2), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(qs=248), -1), (dict(os_=260), -1), (dict(q=p + 2), -1),
                   (dict(H=0), -1), (dict(H=1 << 20), -1), (dict(k=None), -1), (dict(ks=120), -1), (dict(vs=132), -1), (dict(off=None), -1),
                   (dict(lead=2), -2), (dict(R=9), -2), (dict(most=-1), -2), (dict(rows=-1), -2),
                   # rows of q and q_out in one another
                   (dict(out=p, os_=512), -1), (dict(out=p + 16), -1), (dict(out=p + 512, qs=512, os_=520), -1),
                   (dict(out=p + 256, qs=512, os_=512), -1), (dict(out=p + 512 * 2 - 256, qs=512, os_=512), -1),
                   # rows of q_out in those of keys or values
                   (dict(k=far), -1), (dict(v=far), -1), (dict(k=far + 3 * 512 + 496), -1), (dict(v=far + 256, ks=512, os_=512, vs=512), -1),
                   (dict(k=far + 1024 - 240, ks=512, os_=512), -1)):
        assert call(**kw) == rc, (kw, L.dspark_last_error())
    for kw in (dict(R=0), dict(rows=0), dict(most=0)):
        assert call(q=None, out=None, k=None, v=None, off=None, **kw) == 0


def test_history_refuses():
    L, p = B.lib(), _fake()

    def hist(**kw):
        f = dict(seen=p, count=p, rows=4, V=100)
        f.update(kw)
        h = B.dspark_history_t(*[f[n] for n, _ in B.dspark_history_t._fields_])
        KEEP.append(h)
        return ctypes.byref(h)
    for kw, rc in ((dict(seen=None), -1), (dict(count=None), -1), (dict(rows=-1), -2), (dict(V=0), -2), (dict(V=(1 << 30) + 1), -3),
                   (dict(seen=p + 4), -1), (dict(count=p + 8), -1)):
        assert L.dspark_history_clear(hist(**kw), p, 2, None, None) == rc, kw
        assert L.dspark_history_add(hist(**kw), p, 2, 3, p, 0, None, None) == rc, kw
    assert L.dspark_history_clear(None, p, 2, None, None) == -1 == L.dspark_history_add(None, p, 2, 3, p, 0, None, None)
    h = hist()
    assert L.dspark_history_clear(h, None, 5, None, None) == -2 == L.dspark_history_clear(h, p, -1, None, None)
    assert L.dspark_history_add(h, p, 5, 3, None, 0, None, None) == -2 == L.dspark_history_add(h, p, 2, -1, p, 0, None, None)
    assert L.dspark_history_add(h, None, 2, 3, p, 0, None, None) == -1
    assert L.dspark_history_clear(h, None, 0, None, None) == 0 == L.dspark_history_add(h, None, 2, 0, p, 0, None, None)
    assert [L.dspark_history_words(v) for v in (-1, 0, 1, 128, 129, 129280)] == [0, 0, 4, 4, 8, 4040]


def test_target_refuses():
    L, p, ws, far = B.lib(), _fake(1 << 14), _fake(4096), _fake(1 << 14)
    h = B.dspark_history_t(p, p, 4, 100)
    KEEP.append(h)
    base = dict(logits=p, logits_stride=100, n_rows=8, V=100, dtype=1, R=4, lead=1, max_new=2, offsets=p, history=ctypes.addressof(h),
                repetition=p, presence=p, frequency=p, ver_tokens=p, anc=None, bias_off=p, bias_tok=p, bias_val=p, allowed=p,
                allowed_row=p, allowed_stride=4, n_nodes=4, n_bias=4, n_allowed=3, reserved=0, target=p, adjusted=None,
                adjusted_stride=0)

    def call(ws=ws, n=None, **kw):
        f = dict(base, **kw)
        c = B.dspark_target_t(*[f[name] for name, _ in B.dspark_target_t._fields_])
        # no workspace where the other arguments are to pass: nothing is launched
        return L.dspark_target_tokens(ctypes.byref(c), None, None, 0, None) if n is None else L.dspark_target_tokens(ctypes.byref(c), None, ws, n, None)
    small = B.dspark_history_t(p, p, 3, 100)
    other = B.dspark_history_t(p, p, 4, 101)
    wide = dict(V=1 << 20, logits_stride=1 << 20, history=None, allowed=None, allowed_row=None)  # several parts a row
    assert call(**wide) == -4
    assert call(n=64, **wide) == -4
    assert call(ws=ws + 8, n=1 << 40, **wide) == -1
    for kw, rc in ((dict(R=-1), -2), (dict(lead=2), -2), (dict(n_rows=-1), -2), (dict(max_new=-1), -2), (dict(max_new=257), -3),
                   (dict(max_new=65, anc=p), -3), (dict(R=8193), -3), (dict(V=0), -2), (dict(V=(1 << 30) + 1), -3), (dict(dtype=3), -1),
                   (dict(dtype=-1), -1), (dict(n_nodes=-1), -2), (dict(n_bias=-1), -2), (dict(n_allowed=-1), -2),
                   (dict(history=ctypes.addressof(small)), -1), (dict(history=ctypes.addressof(other)), -1), (dict(logits=None), -1),
                   (dict(offsets=None), -1), (dict(target=None), -1), (dict(logits=p + 1), -1), (dict(logits=p + 2, dtype=0), -1),
                   (dict(logits_stride=99), -1), (dict(logits_stride=1 << 62), -1), (dict(adjusted=far, adjusted_stride=99), -1),
                   (dict(adjusted=far + 1, adjusted_stride=100), -1), (dict(adjusted=p, adjusted_stride=100), -1),
                   (dict(adjusted=p + 1598, adjusted_stride=100), -1), (dict(bias_tok=None), -1), (dict(bias_val=None), -1),
                   (dict(allowed_stride=3), -1), (dict(allowed=p + 2), -1), (dict(allowed_row=None, n_allowed=7), -1), (dict(allowed=None), -1)):
        assert call(**kw) == rc, (kw, L.dspark_last_error())
    for kw in (dict(R=0), dict(n_rows=0), dict(max_new=0)):
        assert call(logits=None, offsets=None, target=None, **kw) == 0
    assert L.dspark_target_tokens(None, None, None, 0, None) == -1
    W = L.dspark_target_workspace_bytes
    assert W(0, 5) == W(5, 0) == W(5, (1 << 30) + 1) == 0
    assert 0 < W(1, 129280) < 1 << 16 and W(2048, 129280) < 1 << 25 and W(8, 1 << 30) >= 8 * 8192 * 16


def test_binding_refuses():
    c = B.PagedCache(1, 4, 16, 2, 64, B.DSPARK_BF16, 3, 5, device="cpu")
    off, q, kv = _i32(4), torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    words = torch.zeros(3, dtype=torch.int64)
    rot = B.Rotary(32, device="cpu")
    assert rot.turns.shape == (16,) and rot.turns.dtype == torch.int64
    with pytest.raises(ValueError, match="frequencies"):
        B.Rotary(32, freq=[1.0], device="cpu")
    with pytest.raises(ValueError, match="scaling"):
        B.Rotary(32, scaling="twice", device="cpu")
    with pytest.raises(B.DSparkError):
        B.Rotary(32, base=0.5, device="cpu")
    h = B.History(3, 100, device="cpu")
    assert h.seen.shape == (3, 2, 4) and h.count.shape == (3, 100) and not h.seen.any()
    with pytest.raises(ValueError, match="seen must be"):
        B.History(3, 100, seen=_i32(3, 2, 3))
    x = torch.zeros((3, 100))
    t = _i32(3)
    calls = {
        "attend": lambda **k: B.dspark_cache_attend_tree(c, 0, q, off, 1, 1, k.get("anc", words), 0.1, q.clone()),
        "rotary": lambda **k: B.dspark_cache_append_rotary(c, 0, rot, k.get("q", q), q.clone(), kv, kv, off, 1, 1, depth=k.get("depth")),
        "merge": lambda **k: B.dspark_tree_merge(k.get("tokens", _i32(6, 4)), None, 2, _i32(3), off, _i32(24), k.get("parent", _i32(27))),
        "plan": lambda **k: B.dspark_tree_plan(_i32(9), off, 1, 4, k.get("depth", _i32(9)), k.get("anc", torch.zeros(9, dtype=torch.int64))),
        "accept": lambda **k: B.dspark_accept_tree(_i32(6), off, k.get("parent", _i32(9)), _i32(9), t, k.get("path", _i32(3, 4)), t),
        "keep": lambda **k: B.dspark_cache_keep_path(c, k.get("path", _i32(3, 4)), k.get("n", t), 1),
        "clear": lambda **k: B.dspark_history_clear(h, k.get("rows")),
        "add": lambda **k: B.dspark_history_add(h, k.get("tokens", _i32(3, 5)), True, rows=k.get("rows")),
        "target": lambda **k: B.dspark_target_tokens(k.get("x", x), off, 1, 1, k.get("target", t), **k.get("kw", {})),
    }
    for name, call in calls.items():  # host memory never reaches a kernel
        with pytest.raises(ValueError, match="not the current GPU"):
            call()
    for name, kw, match in (
            ("attend", dict(anc=None), "anc is needed"), ("attend", dict(anc=words[:2]), "2 words for 3"),
            ("attend", dict(anc=words.int()), "int64"), ("rotary", dict(q=q[:2]), "as many rows"),
            ("rotary", dict(depth=_i32(2)), "2 entries"), ("rotary", dict(q=q.half()), "must be"), ("merge", dict(tokens=_i32(5, 4)), "S = 2"),
            ("merge", dict(parent=_i32(26)), "room for"), ("plan", dict(depth=_i32(8)), "each of 9"), ("plan", dict(anc=_i32(9)), "int64"),
            ("accept", dict(parent=_i32(8)), "each of 6"), ("accept", dict(path=_i32(12)), "path must be"),
            ("keep", dict(path=_i32(4, 4)), "at most 3"), ("keep", dict(n=_i32(2)), "accept_len"), ("add", dict(tokens=_i32(5)), "width"),
            ("add", dict(rows=_i32(2)), "rows must be"), ("clear", dict(rows=words), "int32"), ("target", dict(x=x.double()), "float32"),
            ("target", dict(x=x.t().contiguous().t()), "densely packed"), ("target", dict(target=_i32(2)), "each of 3"),
            ("target", dict(kw=dict(penalties=(_i32(3), None, None))), "float32"),
            ("target", dict(kw=dict(penalties=(torch.zeros(2), None, None))), "penalties must be"),
            ("target", dict(kw=dict(bias=(_i32(3), t, t.float()))), "bias_off must be"),
            ("target", dict(kw=dict(allowed=_i32(3, 4).t())), "densely packed"),
            ("target", dict(kw=dict(adjusted=x.half())), "as logits are")):
        with pytest.raises(ValueError, match=match):
            calls[name](**kw)


@pytest.mark.parametrize("dim", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0),
                                dict(scaling="bands", factor=8.0, original=8192.0, low=1.0, high=4.0),
                                dict(scaling="ramp", factor=16.0, original=4096.0, low=1.0, high=32.0),
                                dict(scaling="ramp", factor=2.0, original=7.0, low=1e-3, high=1e3)])
def test_frequencies(dim, kw):
    # pow, log and a handful of products: a few units in the last place
    for base in (10000.0, 500000.0, 1.5):
        np.testing.assert_allclose(B.rotary_frequencies(dim, base, **kw), ot.frequencies(dim, base, **kw), rtol=1e-13)


def test_frequencies_refuse():
    L, p = B.lib(), _fake(4096)

    def call(how=3, dim=64, base=1e4, factor=2.0, original=4096.0, low=1.0, high=32.0, out=p):
        return L.dspark_rotary_frequencies(how, dim, base, factor, original, low, high, out)
    assert call() == 0
    for kw, rc in ((dict(out=None), -1), (dict(dim=0), -1), (dict(dim=7), -1), (dict(how=4), -1), (dict(how=-1), -1), (dict(base=1.0), -2),
                   (dict(base=math.nan), -2), (dict(factor=0.5), -2), (dict(factor=math.inf), -2), (dict(original=0.0), -2), (dict(low=0.0), -2),
                   (dict(low=32.0), -2), (dict(high=math.nan), -2), (dict(original=math.nan), -2)):
        assert call(**kw) == rc, kw
    assert call(how=0, factor=0.0, original=0.0, low=0.0, high=0.0) == 0
    T = L.dspark_rotary_turns
    assert T(None, 0, None) == 0 and T(None, 3, p) == -1 == T(p, 3, None) and T(p, -1, p) == -2
    with pytest.raises(B.DSparkError):
        B.Rotary(4, freq=[1.0, math.inf], device="cpu")


def test_turns_are_exact():
    # 2^64 times the fraction of a turn, off by the division's and the constant's rounding: 2^-63 of a frequency
    freq = [1.0, 0.1, 1e-9, 6.5, 1000.25, -0.3, 0.0] + B.rotary_frequencies(64, 500000.0).tolist()
    turns = np.zeros(len(freq), np.uint64)
    assert B.lib().dspark_rotary_turns((ctypes.c_double * len(freq))(*freq), len(freq), turns.ctypes.data_as(ctypes.c_void_p)) == 0
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")
    for f, got in zip(freq, turns.tolist()):
        want = Fraction(f) / two_pi % 1
        far = abs(Fraction(got, 1 << 64) - want)
        assert min(far, 1 - far) <= Fraction(max(abs(f), 1.0)) / (1 << 63)


def test_binding_refuses_masks_narrower_than_the_vocabulary():
    # a mask's words, not only how far its rows lie apart: the kernel reads ceil(V / 32) of each
    off, t = _i32(5), _i32(4)
    for V, words in ((7000, 10), (7000, 218), (33, 1), (32, 0)):
        x, big = torch.zeros((4, V)), _i32(4, 1000)
        for allowed, match in ((big[:, 1000 - words:], "words"), (big[:1, :words], "words"), (_i32(4, words), "words"),
                               (_i32(0, words), "words"), (big[:, :(V + 31) // 32], "not the current GPU"), (big, "not the current GPU")):
            with pytest.raises(ValueError, match=match):
                B.dspark_target_tokens(x, off, 1, 1, t, allowed=allowed)


def test_a_target_workspace_serves_every_smaller_call():
    # what is promised: rows and tokens up to those that the size was asked for
    L, p, ws = B.lib(), _fake(1 << 14), _fake(4096)
    W = L.dspark_target_workspace_bytes
    sizes = sorted({1, 2, 255, 256, 4095, 4096, 4097, 8193, 100000, 129280, 131072, 131073, 262145}
                   | {512 * 4096 + d for d in (-4096, -1, 0, 1, 255, 256, 257, 4096, 100000)}
                   | {512 * 131072 + d for d in (-1, 0, 1, 131072)} | {513 * 4352, 3 << 20, 1 << 22, (1 << 22) + 1, 1 << 30})
    for n in (1, 2, 3, 100, 4096, 4097, 100000):
        got = [W(n, V) for V in sizes]
        assert got == sorted(got) and got[0] > 0, (n, got)
        assert all(W(n, V) <= W(n + 1, V) for V in sizes)

    def call(V, rows, n):  # the workspace is not aligned, so that one which is large enough is refused for that
        c = B.dspark_target_t(logits=p, logits_stride=V, n_rows=rows, V=V, dtype=1, R=rows, lead=1, max_new=1, offsets=p, target=p)
        return L.dspark_target_tokens(ctypes.byref(c), None, ws + 8, n, None)
    for large in sizes:
        for V in sizes:
            if V <= large:
                for rows in (1, 2, 3, 100, 600, 4097):
                    assert call(V, rows, W(rows, large)) == -1, (V, large, rows)
                assert call(V, 3, W(100, large)) == -1


def test_more_than_a_launch_holds_is_refused():
    # a launch has fewer than 2^32 threads along the requests (rows of tokens), 1024 or 512 to each
    L, p, ws = B.lib(), _fake(1 << 14), _fake(4096)
    h = B.dspark_history_t(p, p, 4, 100)
    KEEP.append(h)
    for n in (1 << 22, (1 << 31) - 1):
        assert L.dspark_history_clear(ctypes.byref(h), p, n, None, None) == -3
        for answered in (0, 1):
            assert L.dspark_history_add(ctypes.byref(h), p, n, 300, p, answered, None, None) == -3

    def target(V, R, rows, ws):
        c = B.dspark_target_t(logits=p, logits_stride=V, n_rows=rows, V=V, dtype=1, R=R, lead=1, max_new=1, offsets=p, target=p)
        return L.dspark_target_tokens(ctypes.byref(c), None, ws, 1 << 40, None)
    assert target(1 << 30, 8192, 1, ws) == -3 == target(1 << 30, 1024, 1024, ws)
    for V, R, rows in ((1 << 30, 1023, 1023), (129280, 8192, 1), (1 << 22, 8192, 1)):  # (not aligned: nothing is launched)
        assert target(V, R, rows, ws + 8) == -1


def test_target_of_rows_without_a_token_is_a_token_or_none():
    L, p, ws = B.lib(), _fake(1 << 14), _fake(4096)

    def call(V, token):
        c = B.dspark_target_t(logits=p, logits_stride=V, n_rows=2, V=V, dtype=1, R=2, lead=1, max_new=1, offsets=p, target=p, reserved=token)
        return L.dspark_target_tokens(ctypes.byref(c), None, ws + 8, 1 << 40, None)  # (not aligned: nothing is launched)
    for V, token, rc in ((100, 0, -1), (100, -1, -1), (100, 99, -1), (1, 0, -1), (100, -2, -2), (100, 100, -2), (1, 1, -2),
                         (100, -(1 << 31), -2), (100, (1 << 31) - 1, -2)):
        assert call(V, token) == rc, (V, token)
