"""CPU checks of the paged cache's entry points: what they refuse, before any HIP call, and
what the binding refuses.  No kernel runs."""
import ctypes

import pytest
import torch

from confidence_scheduled_verification_amd import binding as B

_KEEP = []


def _fake(n=64, align=16):
    # host memory standing in for device pointers: every call below fails its checks first
    buf = (ctypes.c_char * (n + align))()
    _KEEP.append(buf)
    at = ctypes.addressof(buf)
    return at + (-at) % align


def _cache(**kw):
    f = dict(k=_fake(), v=_fake(), table=_fake(), len=_fake(), ref=_fake(), layers=2, n_pages=100, page_size=16,
             n_kv_heads=2, head_dim=64, dtype=1, rows=8, width=10)
    f.update(kw)
    c = B.dspark_cache_t(*[f[n] for n, _ in B.dspark_cache_t._fields_])
    _KEEP.append(c)
    return ctypes.byref(c)


BOOKS = [(dict(n_pages=0), -3), (dict(n_pages=(1 << 24) + 1), -3), (dict(page_size=8), -3), (dict(page_size=48), -3),
         (dict(page_size=512), -3), (dict(rows=-1), -3), (dict(width=0), -3), (dict(rows=1 << 20, width=1 << 12), -3),
         (dict(table=None), -1), (dict(len=None), -1), (dict(ref=None), -1)]
DATA = BOOKS + [(dict(k=None), -1), (dict(v=None), -1), (dict(layers=0), -1), (dict(dtype=0), -3), (dict(dtype=3), -3),
                (dict(head_dim=96), -3), (dict(n_kv_heads=0), -3), (dict(k=_fake() + 8), -1)]


def test_bookkeeping_refuses():
    L, p, ws = B.lib(), _fake(), _fake(4096)
    big = 1 << 20
    for kw, rc in BOOKS:
        c = _cache(**kw)
        assert L.dspark_pages_reserve(c, p, 1, 4, p, None, ws, big, None) == rc, kw
        assert L.dspark_pages_trim(c, p, 4, p, None, None) == rc, kw
        assert L.dspark_pages_commit(c, p, 1, 4, None, None) == rc, kw
    c = _cache(k=None, v=None)  # the books need no contents
    assert L.dspark_pages_reserve(None, p, 1, 4, p, None, ws, big, None) == -1
    assert b"NULL cache" in L.dspark_last_error()
    assert L.dspark_pages_reserve(c, None, 1, 4, p, None, ws, big, None) == -1
    assert L.dspark_pages_reserve(c, p, 1, 4, None, None, ws, big, None) == -1
    assert L.dspark_pages_reserve(c, p, 2, 4, p, None, ws, big, None) == -2
    assert L.dspark_pages_reserve(c, p, 1, 9, p, None, ws, big, None) == -2
    assert L.dspark_pages_reserve(c, p, 1, -1, p, None, ws, big, None) == -2
    assert L.dspark_pages_reserve(_cache(rows=9000), p, 1, 8193, p, None, ws, big, None) == -3
    assert L.dspark_pages_reserve(c, p, 1, 4, p, None, None, 0, None) == -4
    assert L.dspark_pages_reserve(c, p, 1, 4, p, None, ws, 16, None) == -4
    assert L.dspark_pages_reserve(c, p, 1, 4, p, None, ws + 4, big, None) == -1
    assert L.dspark_pages_trim(c, None, 9, None, None, None) == -2
    assert L.dspark_pages_trim(c, p, -1, None, None, None) == -2
    assert L.dspark_pages_commit(c, None, 1, 4, None, None) == -1
    assert L.dspark_pages_commit(c, p, 1, 9, None, None) == -2
    # nothing to do is no error
    assert L.dspark_pages_reserve(c, None, 1, 0, None, None, None, 0, None) == 0
    assert L.dspark_pages_trim(c, p, 0, None, None, None) == 0
    assert L.dspark_pages_commit(c, None, 1, 0, None, None) == 0


def test_moving_pages_refuses():
    L, p, ws = B.lib(), _fake(), _fake(4096)
    big = 1 << 20
    for kw, rc in DATA:
        c = _cache(**kw)
        assert L.dspark_pages_fork(c, p, p, 4, 0, p, None, ws, big, None) == rc, kw
        assert L.dspark_pages_compact(c, p, p, None, ws, big, None) == rc, kw
    c = _cache()
    for args in ((None, p, 4, 0, p), (p, None, 4, 0, p), (p, p, 4, 0, None)):
        assert L.dspark_pages_fork(c, *args, None, ws, big, None) == -1
    assert L.dspark_pages_fork(c, p, p, -1, 0, p, None, ws, big, None) == -2
    assert L.dspark_pages_fork(c, p, p, 8193, 0, p, None, ws, big, None) == -3
    assert L.dspark_pages_fork(_cache(rows=8, width=1 << 20), p, p, 4096, 0, p, None, ws, big, None) == -3
    assert L.dspark_pages_fork(c, p, p, 4, 0, p, None, ws, 64, None) == -4
    assert L.dspark_pages_fork(c, None, None, 0, 0, None, None, None, 0, None) == 0
    assert L.dspark_pages_compact(c, None, p, None, ws, big, None) == -1
    assert L.dspark_pages_compact(c, p, None, None, ws, big, None) == -1
    assert L.dspark_pages_compact(c, p, p, None, None, 0, None) == -4
    assert B.lib().dspark_pages_workspace_bytes(0, 4) == 0 == B.lib().dspark_pages_workspace_bytes(5, -1)


def test_append_refuses():
    L, p = B.lib(), _fake()

    def call(c=None, layer=0, k=p, ks=128, v=p, vs=128, rows=4, off=p, lead=1, R=4, most=8):
        return L.dspark_cache_append(c or _cache(), layer, k, ks, v, vs, rows, off, lead, R, most, None, None)
    for kw, rc in DATA:
        assert call(_cache(**kw)) == rc, kw
    for kw, rc in ((dict(layer=-1), -2), (dict(layer=2), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(ks=120), -1),
                   (dict(vs=132), -1), (dict(k=p + 8), -1), (dict(rows=-1), -2), (dict(off=None), -1), (dict(lead=2), -2),
                   (dict(R=9), -2), (dict(most=-1), -2), (dict(ks=1 << 40), -1)):
        assert call(**kw) == rc, kw
    for kw in (dict(R=0), dict(rows=0), dict(most=0)):
        assert call(k=None, v=None, off=None, **kw) == 0


def test_attend_refuses():
    L, p, ws = B.lib(), _fake(), _fake(4096)
    big = 1 << 40

    def call(c=None, layer=0, q=p, qs=256, rows=4, H=4, off=p, lead=1, R=4, most=8, scale=0.125, ng=0, go=None, st=None,
             sw=0, sp=None, out=p, os_=256, ws=ws, n=big):
        return L.dspark_cache_attend(c or _cache(), layer, q, qs, rows, H, off, lead, R, most, scale, ng, go, st, sw, sp,
                                     out, os_, None, None, ws, n, None)
    for kw, rc in DATA:
        assert call(_cache(**kw)) == rc, kw
    for kw, rc in ((dict(layer=2), -2), (dict(q=None), -1), (dict(out=None), -1), (dict(qs=248), -1), (dict(os_=260), -1),
                   (dict(q=p + 2), -1), (dict(H=3), -1), (dict(H=0), -1), (dict(H=1 << 20), -1), (dict(rows=-1), -2),
                   (dict(off=None), -1), (dict(lead=-1), -2), (dict(R=9), -2), (dict(most=-1), -2), (dict(scale=0.0), -2),
                   (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2),
                   (dict(scale=3.4e38), -2), (dict(ng=-1), -3), (dict(ng=1025), -3), (dict(ng=1), -1),
                   (dict(ng=1, go=p, st=p, sw=0, sp=p), -1), (dict(ws=None), -4), (dict(n=1000), -4), (dict(ws=ws + 8), -1),
                   (dict(rows=1 << 30, most=1 << 29), -3), (dict(c=_cache(width=1 << 28, rows=8, page_size=16)), -3),
                   (dict(ng=1, go=p, st=p, sw=1 << 28, sp=p), -3)):
        assert call(**kw) == rc, (kw, L.dspark_last_error())
    for kw in (dict(R=0), dict(rows=0), dict(most=0)):
        assert call(q=None, out=None, off=None, ws=None, **kw) == 0
    assert L.dspark_cache_attend_workspace_bytes(0, 4, 64, 8, 0) == 0
    one, two = (L.dspark_cache_attend_workspace_bytes(4, 4, 64, 8, g) for g in (0, 1))
    assert 0 < one < two


def test_binding_refuses():
    c = B.PagedCache(1, 4, 16, 2, 64, B.DSPARK_BF16, 3, 5, device="cpu")
    assert c.k.shape == (1, 4, 2, 1, 8, 16, 8) and c.v.shape == (1, 4, 2, 1, 64, 16)
    assert (c.table == -1).all() and (c.len == -1).all() and not c.ref.any()
    books = B.PagedCache(1, 4, 16, 1, 64, B.DSPARK_F16, 3, 5, device="cpu", data=False)
    assert books.k is None and books.v is None
    for args in ((1, 4, 16, 2, 64, B.DSPARK_F32, 3, 5), (1, 4, 20, 2, 64, 1, 3, 5), (0, 4, 16, 2, 64, 1, 3, 5)):
        with pytest.raises(ValueError):
            B.PagedCache(*args, device="cpu")
    with pytest.raises(ValueError, match="table must be"):
        B.PagedCache(1, 4, 16, 2, 64, 1, 3, 5, table=torch.zeros((3, 4), dtype=torch.int32))
    off, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.int32)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not the current GPU"):  # host memory never reaches a kernel
        B.dspark_cache_attend(c, 0, q, off, 1, 1, 0.1, q.clone(), ws=ws)
    with pytest.raises(ValueError, match="not the current GPU"):
        B.dspark_cache_append(c, 0, kv, kv, off, 1, 1)
    for call in (lambda: B.dspark_pages_reserve(c, off, 1, off[:3], ws), lambda: B.dspark_pages_trim(c),
                 lambda: B.dspark_pages_commit(c, off[:3], 1), lambda: B.dspark_pages_fork(c, off, off, off, ws),
                 lambda: B.dspark_pages_compact(c, off, off[:1], ws)):
        with pytest.raises(ValueError, match="not the current GPU"):
            call()
    with pytest.raises(ValueError, match="must be"):
        B.dspark_cache_attend(c, 0, q.half(), off, 1, 1, 0.1, q, ws=ws)
    with pytest.raises(ValueError, match="as many rows"):
        B.dspark_cache_attend(c, 0, q, off, 1, 1, 0.1, q[:2], ws=ws)
    with pytest.raises(ValueError, match="densely packed"):
        B.dspark_cache_attend(c, 0, q.transpose(0, 1).contiguous().transpose(0, 1), off, 1, 1, 0.1, q, ws=ws)
    with pytest.raises(ValueError, match="lse must be"):
        B.dspark_cache_attend(c, 0, q, off, 1, 1, 0.1, q, lse=torch.zeros(3, 3), ws=ws)
    with pytest.raises(ValueError, match="group_off must be"):
        B.dspark_cache_attend(c, 0, q, off, 1, 1, 0.1, q, ws=ws, shared=(off, off.view(2, 2), off[:2]))
    with pytest.raises(ValueError, match="offsets must be"):
        B.dspark_pages_reserve(c, torch.zeros(5, dtype=torch.int32), 1, off, ws)
    with pytest.raises(ValueError, match="contiguous int32"):
        B.dspark_pages_commit(c, off[:3].long(), 1)
    with pytest.raises(ValueError, match="granted must be"):
        B.dspark_pages_reserve(c, off, 1, off, ws)


def test_commit_with_granted_refuses():
    L, p = B.lib(), _fake()
    for kw, rc in BOOKS:
        assert L.dspark_pages_commit_granted(_cache(**kw), p, p, 1, 4, None, None) == rc, kw
    c = _cache(k=None, v=None)
    assert L.dspark_pages_commit_granted(None, p, p, 1, 4, None, None) == -1
    assert L.dspark_pages_commit_granted(c, None, p, 1, 4, None, None) == -1
    assert L.dspark_pages_commit_granted(c, p, p, 1, 9, None, None) == -2
    assert L.dspark_pages_commit_granted(c, p, p, 3, 4, None, None) == -2
    assert L.dspark_pages_commit_granted(c, None, None, 1, 0, None, None) == 0
    books = B.PagedCache(1, 4, 16, 1, 64, B.DSPARK_F16, 3, 5, device="cpu", data=False)
    n = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="granted must be"):
        B.dspark_pages_commit(books, n, 1, granted=n[:2])
    with pytest.raises(ValueError, match="contiguous int32"):
        B.dspark_pages_commit(books, n, 1, granted=n.float())
    with pytest.raises(ValueError, match="not the current GPU"):
        B.dspark_pages_commit(books, n, 1, granted=n)


def test_attend_refuses_tables_that_32_bit_positions_do_not_hold():
    # (no workspace, so that a call that passes the checks of sizes still launches nothing)
    L, p = B.lib(), _fake()

    def call(width, page, shared_width=0):
        groups = (1, p, p, shared_width, p) if shared_width else (0, None, None, 0, None)
        return L.dspark_cache_attend(_cache(width=width, page_size=page, rows=1), 0, p, 256, 4, 4, p, 1, 1, 8, 0.125, *groups,
                                     p, 256, None, None, None, 0, None)
    for page in (16, 256):
        most = ((1 << 31) - 8192) // page
        assert call(most, page) == -4
        assert call(most + 1, page) == call((1 << 31) // page - 1, page) == -3
        assert call(1, page, most) == -4
        assert call(1, page, most + 1) == call(1, page, (1 << 31) // page - 1) == -3


def test_attend_prices_the_work_by_the_form_that_does_it():
    # long prompts over long tables fit; more units than 32 bits number do not (no workspace: nothing runs)
    L, p = B.lib(), _fake()

    def call(rows, H, Hkv, tokens, D=128, groups=0, R=1, most=None):
        c = _cache(width=tokens // 16, rows=R, n_kv_heads=Hkv, head_dim=D)
        g = (groups, p, p, tokens // 16, p) if groups else (0, None, None, 0, None)
        return L.dspark_cache_attend(c, 0, p, H * D, rows, H, p, 1, R, most or rows, 0.125, *g, p, H * D, None, None, None, 0, None)
    assert call(131072, 64, 8, 1 << 20) == -4          # one prompt, a table of a million tokens
    assert call(131072, 32, 2, 1 << 20) == -4          # sixteen heads to a key head
    assert call(131072, 64, 8, 1 << 20, groups=1) == -4
    assert call(300, 64, 8, 1 << 21, R=256, most=(1 << 31) - 1) == -4   # a bound that says nothing
    assert call(1 << 20, 64, 8, 1 << 24) == -3
    assert call(1 << 20, 64, 8, 1 << 24, groups=1) == -3
    assert call(1 << 25, 64, 8, 1 << 20) == -3         # more columns than 2^31
    assert call(1 << 20, 64, 1, 1 << 16, D=256, groups=1) == call(1 << 20, 64, 1, 1 << 16, D=256, groups=1, R=2) == -3


def test_attend_needs_the_workspace_of_its_rows():
    # 255 single tokens and a prompt of 4096 rows behind a prefix (a workspace that is large enough
    # but not aligned is refused as such, so that nothing runs)
    L, p, R, H, n = B.lib(), _fake(), 256, 64, 4351
    c = _cache(rows=R, n_kv_heads=8, head_dim=128, width=600)

    def call(nbytes, max_new=4096, rows=n):
        return L.dspark_cache_attend(c, 0, p, H * 128, rows, H, p, 1, R, max_new, 0.125, 1, p, p, 4, p, p, H * 128, None, None,
                                     p + 8, nbytes, None)
    few, many = (L.dspark_cache_attend_workspace_bytes(*a, 1) for a in ((n, H, 128, 1), (R, H, 128, 4096)))
    assert few < 1 << 30 and many > 1 << 36
    assert call(few) == -1 and b"aligned" in L.dspark_last_error()
    assert call(few, rows=2 * n) == -4 and call(1 << 20) == -4
    assert call(many, rows=R * 4096) == -1
    # sizes whose product passes 64 bits do not wrap round to a few bytes
    assert L.dspark_cache_attend_workspace_bytes(8192, 65535, 256, (1 << 31) - 1, 1) > 1 << 50
    cpu = B.PagedCache(1, 4, 16, 8, 128, B.DSPARK_BF16, R, 5, device="cpu", data=False)
    assert B.cache_workspace(cpu, 4, H, 100, 1, n_rows=103).numel() * 4 < B.cache_workspace(cpu, 4, H, 100, 1).numel() * 4
    assert B.cache_workspace(cpu, 4, H, 3, 1, n_rows=103).numel() == B.cache_workspace(cpu, 4, H, 3, 1).numel()


def test_a_cache_without_rows():
    # its table and lengths are empty (pages that the caller alone holds can be made compact)
    L, p = B.lib(), _fake()
    c = _cache(rows=0, table=None, len=None)
    assert L.dspark_pages_reserve(c, None, 1, 0, None, None, None, 0, None) == 0
    assert L.dspark_pages_trim(c, None, 0, None, None, None) == 0
    assert L.dspark_pages_commit(c, None, 1, 0, None, None) == 0
    assert L.dspark_pages_compact(c, p, p, None, None, 0, None) == -4  # its workspace, no more
    assert L.dspark_pages_trim(c, None, 1, None, None, None) == -2
    assert L.dspark_pages_reserve(c, p, 1, 1, p, None, p, 1 << 20, None) == -2
    assert L.dspark_pages_reserve(_cache(rows=0, table=None, len=None, ref=None), None, 1, 0, None, None, None, 0, None) == -1
