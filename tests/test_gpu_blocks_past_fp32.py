"""Blocks whose scale is past 2^120, the largest that a call sets: what an append that joins one and an eviction make of
their codes."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from tests.blocks_testutil import BlockBatch, stored
from tests.pages_testutil import f64
from tests.test_gpu_evict_scales import cut

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


@pytest.mark.parametrize("old", [2.0 ** 119, 2.0 ** 120, 1.5 * 2.0 ** 120, 2.0 ** 121, 2.0 ** 127, 1.99 * 2.0 ** 127])
def test_append_joins_a_block_of_any_finite_scale(kda, old):
    """A scale is at most 2^120, under which every fp32 value lies within 448: earlier codes that stand for more than
    fp32 holds end at 448."""
    b = BlockBatch(64, 16, Hq=2, Hkv=2, page=32, pos=[9, 25], counts=[2, 3], seed=42)
    for pages, scale in ((b.k_pages, b.k_scale), (b.v_pages, b.v_scale)):
        scale.fill_(old)
        codes = np.random.default_rng(1).integers(0, 256, pages.shape).astype(np.uint8)
        pages.view(torch.uint8).copy_(torch.from_numpy(codes))
    was = f64(b.k_pages), f64(b.v_pages)
    kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=b.T)
    s = min(2.0 ** np.ceil(np.log2(old)), 2.0 ** 120)
    f = float(np.float32(old)) / s
    for pages, scale, before in ((b.k_pages, b.k_scale, was[0]), (b.v_pages, b.v_scale, was[1])):
        for i, page in enumerate((b.np_table()[0][0], b.np_table()[1][0])):
            first = 9 if i == 0 else 25
            begin = first // 16 * 16
            assert (scale[page, :, begin // 16] == s).all()
            got = f64(pages)[page, :, begin:first]
            want = before[page, :, begin:first] * f
            if f in (0.5, 1, 2, 128):
                assert np.array_equal(got, stored(want), equal_nan=True)
            else:  # the product is rounded to fp32 first
                d = np.abs(got - np.clip(want, -448, 448))
                nan = np.isnan(want)
                assert np.array_equal(nan, np.isnan(got))
                assert (d[~nan] <= (2.0 ** -4 + 2.0 ** -23) * np.abs(want[~nan]) + 2.0 ** -10).all()
    assert b.err.item() == 0


@pytest.mark.parametrize("exps", [[121], [124], [127], [-3, 120, 125], [110, 127]])
@pytest.mark.parametrize("codes", [[0x00, 0x80], list(range(0x7f)), [0x40, 0xfe, 0x00, 0x01]])
def test_evict_blocks_of_any_finite_scale(kda, monkeypatch, exps, codes):
    least = mo.block_scale
    monkeypatch.setattr(mo, "block_scale", lambda m: min(least(m), 2.0 ** 120))
    c = cut(exps, codes, 43)
    c.run(kda, 5)
    c.check(5)
