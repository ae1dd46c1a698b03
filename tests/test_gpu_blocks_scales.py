"""Scales by blocks that no append sets, in the attention."""

from __future__ import annotations

import pytest
import torch

from tests.blocks_testutil import BlockBatch
from tests.pages_testutil import check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("width,pos,T,window,dark,rows", [
    (64, 94, 4, 0, 96, [0, 1]),       # the third draft's block and on: the first two rows end before it
    (128, 95, 16, 0, 96, [0]),
    (128, 5001, 8, 0, 5008, list(range(7))),
    (64, 110, 6, 16, 95, [1, 2, 3, 4, 5]),   # a block that only the first row's window reaches
    (128, 2000, 3, 1986, 15, [1, 2]),
    (64, -2, 4, 0, 0, [0, 1])])              # rows before the first token
def test_attend_scales_that_only_some_rows_see(kda, bad, side, width, pos, T, window, dark, rows):
    """A row does not see a block: its scale does not reach it, whatever it is, while other rows of the call see it."""
    b = BlockBatch(width, 16, Hq=8, Hkv=2, page=32, pos=[pos], counts=[T], seed=41)
    ref = b.attend_ref(window=window)
    scale = b.k_scale if side == "k" else b.v_scale
    scale[int(b.np_table()[0][dark // 32]), :, dark % 32 // 16] = bad
    o, lse = b.attend(kda, window=window)
    check_attend(o[rows], lse[rows], [x[rows] for x in ref], b.dt, b.dk, pos + T)
    others = [r for r in range(T) if r not in rows]
    assert not torch.isfinite(o[others]).all()
    assert b.err.item() == 0
