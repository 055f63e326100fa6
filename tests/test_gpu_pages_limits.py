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
