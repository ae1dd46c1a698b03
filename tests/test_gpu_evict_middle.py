"""The choice of rows that one workgroup reads again for every pass: longer than it holds in registers, and too short or
too many to be shared out to several."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_evict import WEIGHTS, Cut

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


@pytest.mark.parametrize("name", WEIGHTS)
@pytest.mark.parametrize("lens,keep,recent", [([8200, 20000, 40000], 300, 40), ([8192, 8193, 8194], 8000, 0),
                                              ([8292, 8293, 16484], 500, 100), ([17409, 33792, 16385], 16000, 1),
                                              ([40000, 100], 1, 0), ([30000], 29999, 7)])
def test_middle_lengths(kda, name, lens, keep, recent):
    """Tables of 8193 to 40960 places; candidates about what registers hold (8192) and at ends of a pass (16384 and on);
    keys that share the first digit few enough for the list of 8192, and not."""
    c = Cut("e4m3_d64", lens, keep, Hkv=1, page=128, seed=5, weights=WEIGHTS[name])
    assert 8192 < c.b.table.shape[1] * 128 <= 40960
    c.run(kda, recent)
    c.check(recent)
    assert c.b.err.item() == 0


@pytest.mark.parametrize("name", ["all equal", "few values", "any sign and size", "infinite and nan"])
def test_many_rows_of_a_long_table(kda, name):
    """More than 32 rows of a table past 40960 places, short and long."""
    lens = [45000, 8193, 12000] + [int(x) for x in np.random.default_rng(1).integers(0, 600, 30)]
    c = Cut("e4m3_d64", lens, 256, Hkv=1, page=128, seed=6, weights=WEIGHTS[name])
    c.run(kda, 20)
    c.check(20)
    assert c.b.err.item() == 0


@pytest.mark.parametrize("tokens", [30000, 60000])
def test_long_rows_captured_and_on_two_streams(kda, tokens):
    """The choice by one workgroup and by several: every replay, and two calls at once, give the eager call's results."""
    lens, keep = [tokens, tokens // 2, 700], 500  # the third is cut at first, and then stays
    a, b, c = (Cut("e4m3_d64", lens, keep, Hkv=2, page=128, seed=9) for _ in range(3))
    plans = [kda.KvEvictPlan(x.b.pool(kda), x.b.table, x.len, x.w, x.dst, x.new_len, x.new_w, x.kept, x.b.err, recent=60)
             for x in (a, b, c)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for p in plans:
        p()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plans[1]()
    for step in range(4):
        for x in (a, b, c):
            x.w.random_(0, 5000, generator=torch.Generator(x.device).manual_seed(step))
            x.len.copy_(torch.tensor([tokens - 3000 * step, tokens // 2 - 100 * step, 700 - 90 * step]))
            x.kept.fill_(7)
        torch.cuda.synchronize()
        for p, s in zip((plans[0], plans[2]), streams):
            with torch.cuda.stream(s):
                p()
        graph.replay()
        torch.cuda.synchronize()
        a.lens = a.len.tolist()
        a.check(60)
        a.before = [None if x is None else x.clone() for x in (a.b.k_pages, a.b.v_pages, a.b.k_scale, a.b.v_scale)]
        for x in (b, c):
            for s, t in ((a.kept, x.kept), (a.new_w, x.new_w), (a.new_len, x.new_len),
                         (a.b.k_pages.view(torch.uint8), x.b.k_pages.view(torch.uint8)),
                         (a.b.v_pages.view(torch.uint8), x.b.v_pages.view(torch.uint8))):
                assert torch.equal(s, t)
    assert a.b.err.item() == b.b.err.item() == c.b.err.item() == 0
