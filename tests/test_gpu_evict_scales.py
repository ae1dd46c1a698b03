"""Eviction into pages with scales by blocks at the ends of their range: zeros stay zeros, and what fp32 cannot hold
counts as its largest value.  Against the fp64 oracle, bit for bit."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_evict import Cut

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def cut(exps, codes, seed, *, width=64, block=16, page=32, lens=(70, 45), keep=20):
    """A Cut whose blocks have scales of 2^exps[..] and whose codes come from `codes` (bytes), drawn for each."""
    c = Cut(f"blocks_d{width}", list(lens), keep, page=page, block=block, seed=seed)
    rng = np.random.default_rng(seed)
    b = c.b
    for pages, scale in ((b.k_pages, b.k_scale), (b.v_pages, b.v_scale)):
        pages.view(torch.uint8).copy_(torch.from_numpy(rng.choice(np.array(codes, np.uint8), pages.shape)))
        scale.copy_(torch.from_numpy(np.float32(2.0) ** rng.choice(np.array(exps, np.float32), scale.shape)))
    c.before = [x.clone() for x in (b.k_pages, b.v_pages, b.k_scale, b.v_scale)]
    return c


ZEROS = [0x00, 0x80]


@pytest.mark.parametrize("exps", [[63], [64], [119], [120], [-64, 0, 64, 120]])
@pytest.mark.parametrize("width,block,page", [(64, 16, 32), (128, 32, 32), (64, 256, 256)])
def test_zeros_stay_zeros(kda, exps, width, block, page):
    """Blocks of zeros whose scale an outlier had raised: the new one is 2^-64, and the factor between them passes fp32."""
    c = cut(exps, ZEROS, 31, width=width, block=block, page=page, lens=(3 * page + 7, 2 * page), keep=page + 5)
    c.run(kda, 4)
    c.check(4)
    assert not torch.isnan(c.b.k_pages.float()).any() and not torch.isnan(c.b.v_pages.float()).any()


@pytest.mark.parametrize("seed", range(4))
def test_rows_of_zeros_beside_small_ones(kda, seed):
    """Each kept row all zeros under a large scale, or small codes under a small one: they share new blocks."""
    c = cut([120], ZEROS, seed)
    b = c.b
    rng = np.random.default_rng(seed + 100)
    for pages, scale in ((b.k_pages, b.k_scale), (b.v_pages, b.v_scale)):
        small = torch.from_numpy(rng.random(scale.shape) < 0.5).to(b.device)
        scale[small] = 2.0 ** -20
        rows = small.repeat_interleave(b.block, 2)
        codes = torch.from_numpy(rng.integers(0, 0x7f, pages.shape).astype(np.uint8)).to(b.device)
        pages.view(torch.uint8)[rows] = codes[rows]
    c.before = [x.clone() for x in (b.k_pages, b.v_pages, b.k_scale, b.v_scale)]
    c.run(kda, 3)
    c.check(3)


@pytest.mark.parametrize("exps", [[120], [118, 119, 120], [-64, 120]])
@pytest.mark.parametrize("codes", [[0x78, 0xf8], [0x77, 0x78, 0x7e, 0x00, 0xfe], list(range(0x7f)) + [0x7f]])
def test_values_past_fp32_count_for_the_scale(kda, exps, codes):
    """256 at a scale of 2^120, which an append of the largest fp32 values stores, is 2^128: the block needs 2^120."""
    c = cut(exps, codes, 37)
    c.run(kda, 5)
    for pages in (c.b.k_pages, c.b.v_pages):  # 0x7f and 0xff are both NaN; which one comes out is left open
        pages.view(torch.uint8)[torch.isnan(pages.float())] = 0x7f
    c.check(5)
