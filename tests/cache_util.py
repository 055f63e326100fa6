"""Helpers of the paged cache's GPU tests: random states, uploads, and the comparison with
the oracle under bounds derived from the arithmetic."""
from __future__ import annotations

import numpy as np
import torch

from confidence_scheduled_verification_amd import binding as B
from oracle import cache as oc

DEV = "cuda"
DT = {"bf16": (B.DSPARK_BF16, torch.bfloat16), "fp16": (B.DSPARK_F16, torch.float16)}


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def rounded(x, dtype):
    """float64 values as the 16-bit type holds them."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype][1])


class State:
    """A cache on the device and its mirror: table, len and ref as lists, K and V in token order."""

    def __init__(self, rng, layers, n_pages, page, heads, D, dtype, rows, width, fill=np.nan):
        self.page, self.dtype = page, dtype
        shape = (layers, n_pages, heads, page, D)
        self.k, self.v = np.full(shape, fill), np.full(shape, fill)
        self.table, self.len, self.ref = [[-1] * width for _ in range(rows)], [0] * rows, [0] * n_pages
        self.cache = B.PagedCache(layers, n_pages, page, heads, D, DT[dtype][0], rows, width, device=DEV)
        self.rng = rng

    def give(self, r, pages):
        """Row r gets as many pages, picked at random from the free ones."""
        free = [p for p, n in enumerate(self.ref) if n == 0]
        for i, p in enumerate(self.rng.permutation(free)[:pages].tolist()):
            self.table[r][i] = p
            self.ref[p] = 1

    def put(self, layer, ids, first, n):
        """Random K and V for n tokens from position `first` of the pages ids on."""
        for x in (self.k, self.v):
            for p in range(first, first + n):
                y = self.rng.standard_normal(x.shape[2:3] + x.shape[4:])
                x[layer, ids[p // self.page], :, p % self.page] = rounded(y, self.dtype).double().numpy()

    def upload(self):
        c = self.cache
        c.table.copy_(i32(self.table).reshape(c.table.shape))
        c.len.copy_(i32(self.len))
        c.ref.copy_(i32(self.ref))
        c.k.copy_(rounded(oc.pack_k(self.k), self.dtype))
        c.v.copy_(rounded(oc.pack_v(self.v), self.dtype))
        return c

    def assert_books(self):
        c = self.cache
        np.testing.assert_array_equal(c.table.cpu().numpy(), np.asarray(self.table, np.int32))
        np.testing.assert_array_equal(c.len.cpu().numpy(), np.asarray(self.len, np.int32))
        np.testing.assert_array_equal(c.ref.cpu().numpy(), np.asarray(self.ref, np.int32))

    def assert_data(self):
        np.testing.assert_array_equal(oc.unpack_k(self.cache.k.cpu().double().numpy()), self.k)
        np.testing.assert_array_equal(oc.unpack_v(self.cache.v.cpu().double().numpy()), self.v)


def attend_bounds(want, dtype, keys, D):
    """How far out and lse may be off, from the roundings alone.
    A score is D products of 16-bit values, exact in fp32, summed there in some order: off by at
    most D 2^-24 of scale sum |q||K| = reach; the scale's and the exponent's own roundings are
    4 2^-24 of the score and of the maximum, 2^-21 covers exp2's two ulps; so each weight is off by
    the relative e = (D + 8) 2^-24 reach + 2^-21, to first order, and the ratio of two sums of up to
    `keys` weights by 2 e + 2 keys 2^-24.  The weights' rounding for the second product is half a
    step u (bf16 2^-8, fp16 2^-11; below fp16's smallest normal half of 2^-24, relative to the
    largest weight of 1), the result's rounding another.  All of that times spread, the weighted
    mean of |V|, which is at least |out|."""
    out, lse, spread, reach = want
    u = float(torch.finfo(DT[dtype][1]).eps) / 2
    e = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
    tiny = keys * 2.0 ** -25 if dtype == "fp16" else 0.0
    rel = 1.05 * (2 * e + 2 * keys * 2.0 ** -24)
    vmax = 8.0  # normal values stay below
    b_out = (rel[..., None] + 1.05 * u) * spread + u * np.abs(out) + tiny * vmax + 2.0 ** -24
    return b_out, rel + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def assert_attend(out, lse, want, dtype, keys, D, left=None):
    """`left`: what rows of no request held before the call."""
    w_out, w_lse, _, reach = want
    b_out, b_lse = attend_bounds(want, dtype, keys, D)
    out = out.detach().cpu().double().numpy()
    lse = None if lse is None else lse.cpu().double().numpy()
    nobody = reach < 0
    some = np.isfinite(w_out) & ~nobody[..., None]
    with np.errstate(invalid="ignore"):
        d = np.abs(out - w_out)
    bad = some & ~(d <= b_out)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), d[bad][:5], b_out[bad][:5])
    special = ~some & ~nobody[..., None]
    np.testing.assert_array_equal(out[special], w_out[special])
    if left is not None:
        assert (out[nobody] == left).all()
    if lse is not None:
        fin = np.isfinite(w_lse) & ~nobody
        with np.errstate(invalid="ignore"):
            bad = fin & ~(np.abs(lse - w_lse) <= b_lse)
        assert not bad.any(), (np.argwhere(bad)[:5].tolist(), lse[bad][:5], w_lse[bad][:5])
        np.testing.assert_array_equal(lse[~fin & ~nobody], w_lse[~fin & ~nobody])
        if left is not None:
            assert (lse[nobody] == left).all()
