"""How the paged attention's work is split: row blocks, tiles, workers' runs and pieces, and the loads that large pools
select."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.pages_testutil import Batch, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


@pytest.mark.parametrize("hq,room", [(16, 512), (32, 1 << 13), (64, 1 << 15), (128, 1 << 18)])
def test_latent_row_blocks_by_number_of_tiles(kda, hq, room):
    """Blocks of 16, 32, 64 and 128 rows over one to nine tiles of 32 tokens, again and again: the same bits."""
    pos = [32 * n - 1 for n in range(1, 10)]
    b = Batch("latent", Hq=hq, Hkv=1, page=64, pos=pos, counts=[1] * 9, seed=51, extra_cols=room // 64 - 5)
    ref = b.attend_ref()
    o, lse = b.attend(kda)
    check_attend(o, lse, ref, b.dt, b.dk, 288)
    for _ in range(5):
        o2, lse2 = b.attend(kda)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert b.err.item() == 0
