"""Books and append of the paged cache at the edges of what their calls allow."""
import numpy as np
import pytest
import torch

import cache_util as cu
from confidence_scheduled_verification_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lead", [0, 1])
def test_a_request_without_rows_appends_nothing(lead):
    # an idle request whose last, partly filled page another row holds too: nothing to flag
    print("append, idle request", lead, flush=True)
    st = cu.State(np.random.default_rng(51), 1, 8, 16, 1, 64, "bf16", 2, 4)
    st.len = [20, 24]
    st.give(0, 2)
    st.table[1][:2] = st.table[0][:2]
    for i in st.table[0][:2]:
        st.ref[i] = 2
    st.put(0, st.table[0], 0, 32)
    c = st.upload()
    before = c.k.clone(), c.v.clone()
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    kn = torch.ones((2, 1, 64), dtype=torch.bfloat16, device=cu.DEV)
    B.dspark_cache_append(c, 0, kn, kn, cu.i32([2, 2 - lead, 2 - 2 * lead]), lead, 2, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, b in zip(before, (c.k, c.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_trim_of_as_many_rows_as_a_grid_has_threads():
    # more rows than 2^32 threads hold at a wave a row
    print("trim, many rows", flush=True)
    rows = (1 << 26) + 5
    c = B.PagedCache(1, 64, 16, 1, 64, B.DSPARK_BF16, rows, 1, device=cu.DEV, data=False)
    c.len.zero_()
    held = [0, 3, (1 << 26) - 1, 1 << 26, rows - 1]
    for p, r in enumerate(held):
        c.table[r, 0], c.len[r], c.ref[p] = p, 9, 1
    keep = torch.full((rows,), 7, dtype=torch.int32, device=cu.DEV)
    keep[3] = keep[rows - 1] = 0
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    B.dspark_pages_trim(c, None, keep, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert c.table[held, 0].tolist() == [0, -1, 2, 3, -1] and c.len[held].tolist() == [7, 0, 7, 7, 0]
    assert c.ref[:5].tolist() == [1, 0, 1, 1, 0] and int((c.len != 0).sum()) == 3


def test_compact_without_rows():
    # pages that the caller alone holds
    print("compact, no rows", flush=True)
    c = B.PagedCache(1, 5, 16, 1, 64, B.DSPARK_BF16, 0, 3, device=cu.DEV)
    c.ref.copy_(cu.i32([0, 1, 0, 0, 2]))
    c.k[0, 4], c.v[0, 4] = 4.0, 5.0
    page_map, n_live = torch.zeros(5, dtype=torch.int32, device=cu.DEV), torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    status = torch.zeros(1, dtype=torch.int32, device=cu.DEV)
    B.dspark_pages_compact(c, page_map, n_live, B.pages_workspace(c, 0), status)
    B.dspark_pages_trim(c)
    torch.cuda.synchronize()
    assert page_map.tolist() == [-1, 1, -1, -1, 0] and n_live.item() == 2 and status.item() == 0
    assert c.ref.tolist() == [2, 1, 0, 0, 0] and (c.k[0, 0] == 4).all() and (c.v[0, 0] == 5).all()
