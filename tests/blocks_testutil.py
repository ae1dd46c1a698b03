"""Seeded caches whose e4m3 pages have scales by blocks, and what the tests of the calls on them expect."""

from __future__ import annotations

import numpy as np
import torch

from oracle import paged_more_oracle as mo
from oracle import paged_oracle as po
from tests.pages_testutil import Batch, f64

E4M3 = torch.float8_e4m3fn


def stored(x):
    """float64 values as e4m3 holds them (rounded to nearest even, from fp32), as float64."""
    y = torch.from_numpy(np.ascontiguousarray(x)).float().clamp(-448, 448).to(E4M3)
    return y.float().numpy().astype(np.float64)


class BlockBatch(Batch):
    """A Batch over pages with scales by blocks: powers of two of a few sizes."""

    def __init__(self, width, block, *, scale_seed=77, exps=(-9, -4), **kw):
        super().__init__(f"e4m3_d{width}", **kw)
        self.block = block
        rng = np.random.default_rng(scale_seed)
        shape = (self.n_pages, self.Hkv, self.page // block)
        self.k_scale, self.v_scale = (
            torch.from_numpy(2.0 ** rng.integers(*exps, shape)).float().to(self.device) for _ in range(2))

    def pool(self, kda):
        return kda.PagePool.from_tensors(self.k_pages, self.v_pages, k_scale=self.k_scale, v_scale=self.v_scale,
                                         scale_block=self.block)

    def values(self):
        return (mo.unscaled(f64(self.k_pages), f64(self.k_scale), self.block),
                mo.unscaled(f64(self.v_pages), f64(self.v_scale), self.block))

    def attend_ref(self, scale=None, window=0, q=None):
        k, v = self.values()
        return po.attend(k, v, self.np_table(), self.pos.cpu().numpy(), self.counts, f64(self.q if q is None else q),
                         self.dk ** -0.5 if scale is None else scale, window, None, None, self.dv)


def check_stored(got, got_scale, before, before_scale, table, pos, counts, rows, block, err, what=""):
    """One side of the pages after an append of `rows` (fp64, rotated; err: how far the kernel's fp32 ones may be off).

    Scales are the formula's exactly (no block's maximum may lie within `err` of a border).  A new value is a rounding
    (half a step, 2^-4 relative, 2^-10 of the scale where subnormal) of an fp32 value within err of x.  Earlier tokens
    are the e4m3 of old * ratio, exactly.  Every other byte is as before.
    """
    want, scales = f64(before), f64(before_scale)
    was = want.copy()
    top = mo.append_blocks(want, scales, table, pos, counts, rows, block)
    for (page, h, k), m in top.items():
        assert mo.block_scale(max(m - err, 0)) == mo.block_scale(m + err), "a block's maximum lies at a border"
    assert np.array_equal(f64(got_scale), scales), f"{what}: scales"
    per, page_size, row = want.shape[2] // block, want.shape[2], 0
    new = np.zeros(want.shape[:3], bool)
    old = np.zeros(want.shape[:3], bool)
    for b, n in enumerate(counts):
        for i in range(n):
            p = int(pos[b]) + i
            new[table[b][p // page_size], :, p % page_size] = True
        if n and pos[b] % block:
            first = int(pos[b]) % page_size
            old[table[b][int(pos[b]) // page_size], :, first // block * block:first] = True
        row += n
    s = np.repeat(scales, block, axis=2)[..., None]
    g = f64(got)
    assert np.array_equal(g[~new & ~old], was[~new & ~old], equal_nan=True), f"{what}: other places"
    assert np.array_equal(g[old], stored(want[old]), equal_nan=True), f"{what}: earlier tokens of a block"
    fin = np.isfinite(want) & new[..., None]
    tol = (np.abs(want) + err / s) * 2.0 ** -4 + 2.0 ** -10 + err / s
    assert (np.abs(g - want)[fin] <= tol[fin]).all(), f"{what}: new values off by {np.abs(g - want)[fin].max()}"
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN"
    assert per >= 1
