"""Eviction from the paged cache on the GPU: places, rows and sums against the oracle, exactly."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from tests.blocks_testutil import BlockBatch, stored
from tests.pages_testutil import FORMS, Batch, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


class Cut:
    """A batch with lengths, weights, and spare pages to move to."""

    def __init__(self, form, lens, keep, *, Hkv=2, page=16, block=16, seed=0, weights=None, extra=3, wide=0):
        kw = dict(Hq=Hkv, Hkv=Hkv, page=page, pos=list(lens), counts=[0] * len(lens), seed=seed, extra_cols=1)
        dst = -(-keep // page)
        spare = dst * len(lens) + extra
        self.blocks = form.startswith("blocks")
        self.b = b = BlockBatch(int(form.split("_d")[1]), block, spare=spare, **kw) if self.blocks else Batch(form, spare=spare, **kw)
        used = set(b.np_table().flatten()) - {-1}
        free = [i for i in range(b.n_pages) if i not in used]
        rng = np.random.default_rng(seed + 1)
        rng.shuffle(free)
        to = np.full((len(lens), dst + wide), -1, np.int32)
        to[:, :dst] = np.array(free[:dst * len(lens)], np.int32).reshape(len(lens), dst)
        dev = self.device = b.device
        self.lens, self.keep = list(lens), keep
        self.len = torch.tensor(self.lens, dtype=torch.int64, device=dev)
        self.dst = torch.from_numpy(to).to(dev)
        w = rng.random((len(lens), Hkv, b.table.shape[1] * page + 3), dtype=np.float32) if weights is None else weights(rng, (len(lens), Hkv, b.table.shape[1] * page + 3))
        self.w = torch.from_numpy(np.asarray(w, np.float32)).to(dev)
        self.new_w = torch.full_like(self.w, 7.0)
        self.kept = torch.full((len(lens), Hkv, keep), 7, dtype=torch.int32, device=dev)
        self.new_len = torch.full((len(lens),), 7, dtype=torch.int64, device=dev)
        self.before = [None if x is None else x.clone() for x in (b.k_pages, b.v_pages, b.k_scale, b.v_scale)]

    def run(self, kda, recent=0, new_len=None):
        kda.kv_evict(self.b.pool(kda), self.b.table, self.len, self.w, self.dst,
                     self.new_len if new_len is None else new_len, self.new_w, self.kept, self.b.err, recent=recent)
        torch.cuda.synchronize()
        assert kda.last_variant() == "kv_evict"

    def check(self, recent=0, refused=()):
        b, keep, w = self.b, self.keep, self.w.cpu().numpy()
        pages = [None if x is None else x.cpu() for x in self.before]
        sides = [0] if b.v_pages is None else [0, 1]
        want = [pages[i].clone().view(torch.uint8) for i in sides]
        scales = [pages[2 + i].clone() for i in sides] if self.blocks else None
        table, dst = b.np_table(), self.dst.cpu().numpy()
        for s, L in enumerate(self.lens):
            stays = s in refused or L <= keep
            assert self.new_len[s].item() == (L if stays else keep)
            for h in range(b.Hkv):
                new_w = np.zeros(w.shape[2], np.float32)
                if stays:
                    assert (self.kept[s, h] == -1).all()
                    if s not in refused:
                        new_w[:L] = w[s, h, :L]
                else:
                    places = np.array(mo.keep_places(w[s, h], L, keep, recent))
                    assert np.array_equal(self.kept[s, h].cpu().numpy(), places), (s, h)
                    new_w[:keep] = w[s, h, places]
                    self.move(want, scales, pages, sides, table[s], dst[s], h, places)
                assert np.array_equal(self.new_w[s, h].cpu().numpy(), new_w, equal_nan=True), (s, h)
        for i in sides:
            got = (b.k_pages, b.v_pages)[i].cpu().view(torch.uint8)
            assert torch.equal(got, want[i]), ("k", "v")[i]
            if self.blocks:
                assert torch.equal((b.k_scale, b.v_scale)[i].cpu(), scales[i])

    def move(self, want, scales, pages, sides, table, dst, h, places):
        page, keep = self.b.page, self.keep
        src = torch.from_numpy(table[places // page]).long(), torch.from_numpy(places % page)
        i = np.arange(keep)
        to = torch.from_numpy(dst[i // page]).long(), torch.from_numpy(i % page)
        for side in sides:
            rows = pages[side].view(torch.uint8)[src[0], h, src[1]]
            if self.blocks:
                block = self.b.block
                x = rows.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
                x = x * pages[2 + side][src[0], h, src[1] // block].numpy().astype(np.float64)[:, None]
                for first in range(0, keep, block):
                    part = x[first:first + block]
                    s = mo.block_scale(np.abs(part[np.isfinite(part)]).max(initial=0.0))
                    scales[side][int(to[0][first]), h, int(to[1][first]) // block] = s
                    y = torch.from_numpy(stored(part / s)).float().to(torch.float8_e4m3fn).view(torch.uint8)
                    want[side][to[0][first:first + block], h, to[1][first:first + block]] = y
            else:
                want[side][to[0], h, to[1]] = rows


@pytest.mark.parametrize("form,recent", itertools.product(list(FORMS) + ["blocks_d64", "blocks_d128"], [0, 5, 20]))
def test_forms(kda, form, recent):
    c = Cut(form, [70, 20, 21, 0, 100], 20, Hkv=1 if form == "latent" else 2, seed=recent)
    c.run(kda, recent)
    c.check(recent)
    assert c.b.err.item() == 0


@pytest.mark.parametrize("keep", [1, 15, 16, 17, 63, 64, 65, 200, 299])
@pytest.mark.parametrize("form", ["bf16_d64", "blocks_d64"])
def test_budgets(kda, form, keep):
    c = Cut(form, [300, keep, keep + 1, 5000], keep, page=64, block=32, seed=keep, wide=2)
    recent = keep // 3
    c.run(kda, recent)
    c.check(recent)


@pytest.mark.parametrize("block,page", [(16, 1024), (64, 64), (128, 256), (256, 256), (256, 1024), (32, 512)])
def test_blocks(kda, block, page):
    c = Cut("blocks_d128", [3000, 1500], 1100, page=page, block=block, seed=block)
    c.run(kda, 100)
    c.check(100)


WEIGHTS = {
    "all equal": lambda rng, shape: np.full(shape, 0.25),
    "zeros": lambda rng, shape: np.zeros(shape),
    "signed zeros": lambda rng, shape: np.where(rng.random(shape) < 0.5, -0.0, 0.0),
    "few values": lambda rng, shape: rng.integers(0, 4, shape) / 4,
    "last bits": lambda rng, shape: np.float32(1) + rng.integers(0, 3, shape).astype(np.float32) * np.float32(2.0 ** -23),
    "any sign and size": lambda rng, shape: rng.standard_normal(shape) * 10.0 ** rng.integers(-40, 30, shape),
    "infinite and nan": lambda rng, shape: np.where(rng.random(shape) < 0.3, np.nan, np.where(
        rng.random(shape) < 0.3, np.inf, np.where(rng.random(shape) < 0.3, -np.inf, rng.random(shape)))),
    "mostly nan": lambda rng, shape: np.where(rng.random(shape) < 0.99, np.nan, 1.0),
}


@pytest.mark.parametrize("name", WEIGHTS)
@pytest.mark.parametrize("recent", [0, 9, 150])
def test_orders(kda, name, recent):
    c = Cut("bf16_d64", [400, 2300, 151], 150, seed=3, weights=WEIGHTS[name])
    c.run(kda, recent)
    c.check(recent)


def test_long_and_many(kda):
    c = Cut("bf16_d64", [70001], 9000, Hkv=2, page=64, seed=4)
    c.run(kda, 777)
    c.check(777)
    c = Cut("e4m3_d64", [int(x) for x in np.random.default_rng(0).integers(0, 90, 150)], 40, Hkv=1, seed=5)
    c.run(kda, 3)
    c.check(3)


@pytest.mark.parametrize("name", WEIGHTS)
@pytest.mark.parametrize("lens,keep,recent", [([50000, 8000, 100], 200, 150), ([41000, 8193, 16384, 30000], 8000, 0),
                                              ([70000], 60000, 60000), ([65536, 65537], 8192, 1)])
def test_long_tables(kda, name, lens, keep, recent):
    """Rows shared out to several workgroups, among them short ones, and parts that end at a row's candidates."""
    c = Cut("e4m3_d64", lens, keep, Hkv=1, page=128, seed=5, weights=WEIGHTS[name])
    c.run(kda, recent)
    c.check(recent)
    assert c.b.err.item() == 0


def test_long_tables_refusals(kda):
    c = Cut("e4m3_d64", [50000, 50000, 45000, 9000], 9000, Hkv=2, page=128, seed=6, extra=0)
    c.b.table[0, 70] = -1
    c.len[1] = c.b.table.shape[1] * 128 + 1
    c.lens[1] = c.len[1].item()
    c.run(kda, 100)
    assert c.b.err.item() == kda.DEV_ERR_PAGE
    c.check(100, refused=(0, 1))


def test_lengths_in_place(kda):
    c = Cut("bf16_d64", [70, 20, 21], 20, seed=6)
    c.run(kda, 5, new_len=c.len)
    assert c.len.tolist() == [20, 20, 20]
    c.new_len = c.len
    c.check(5)


def test_refusals(kda):
    """Lengths outside the table and bad pages leave their sequence alone."""
    c = Cut("blocks_d64", [70, 60, 50, 40, 30, 10], 20, seed=7, extra=0)
    c.b.table[1, 1] = c.b.n_pages
    c.dst[2, 1] = -1
    c.len[3], c.len[4] = -1, c.b.table.shape[1] * 16 + 1
    c.lens[3], c.lens[4] = -1, c.b.table.shape[1] * 16 + 1
    c.b.table[5, 0] = -7                              # a short sequence: not looked at
    c.run(kda, 4)
    assert c.b.err.item() == kda.DEV_ERR_PAGE
    c.check(4, refused=(1, 2, 3, 4))


def test_on_another_stream_and_replayed(kda):
    a, b = (Cut("blocks_d128", [70, 200], 40, seed=8) for _ in range(2))
    plans = [kda.KvEvictPlan(x.b.pool(kda), x.b.table, x.len, x.w, x.dst, x.new_len, x.new_w, x.kept, x.b.err, recent=3)
             for x in (a, b)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        plans[0]()
    torch.cuda.synchronize()
    a.check(3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plans[1]()
    for step in range(4):
        for x in (a, b):
            x.w.random_(0, 50, generator=torch.Generator(x.device).manual_seed(step))
            x.len.copy_(torch.tensor([70 - 8 * step, 200 - 60 * step]))
        plans[0]()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((a.kept, b.kept), (a.new_w, b.new_w), (a.new_len, b.new_len), (a.b.k_scale, b.b.k_scale),
                     (a.b.k_pages.view(torch.uint8), b.b.k_pages.view(torch.uint8)),
                     (a.b.v_pages.view(torch.uint8), b.b.v_pages.view(torch.uint8))):
            assert torch.equal(x, y)


@pytest.mark.parametrize("form", ["bf16_d128", "blocks_d128"])
def test_a_serving_loop(kda, form):
    """Decode rounds with explicit positions, sums of weights, and two evictions: append, attend, weigh, cut, go on.

    The attention after a cut sees the kept tokens: against fp64 attention over the rows that were appended (rounded as
    stored), at the places that `kept` names."""
    dev, B, Hq, Hkv, d, page, keep, recent = "cuda", 2, 4, 2, 128, 16, 20, 6
    blocks = form.startswith("blocks")
    g = torch.Generator(dev).manual_seed(1)
    pool = kda.PagePool(40, page, Hkv, d, d, dev, dtype=torch.float8_e4m3fn if blocks else torch.bfloat16,
                        scale_block=16 if blocks else 0)
    tables = torch.arange(2 * B * 4, dtype=torch.int32, device=dev).view(2, B, 4)   # two sets of pages, used in turn
    ang = torch.arange(200)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    place = torch.zeros(B, dtype=torch.int64, device=dev)
    at = torch.zeros(B, dtype=torch.int64, device=dev)      # positions go on where places are cut
    weights = torch.zeros((B, Hkv, 64), device=dev)
    ws = kda.attn_workspace(pool, tables[0], Hq=Hq, T=4)
    rows = [[[] for _ in range(Hkv)] for _ in range(B)]     # what each head's cache holds: (key, value) in fp64
    turn = 0
    for step in range(20):
        T = 4 if step % 3 == 0 else 1
        q, k, v = (torch.randn((B, T, h, d), device=dev, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        axis_pos = (at[:, None] + torch.arange(T, device=dev))[None].contiguous()
        q_rot = torch.empty_like(q)
        kda.kv_append(pool, tables[turn], place, k, v, err, q=q, q_out=q_rot, cos_sin=cos_sin, axis_pos=axis_pos)
        o, lse = torch.empty_like(q), torch.empty((B, T, Hq), device=dev)
        kda.attn_decode(pool, tables[turn], place, q_rot, o, ws, err, lse=lse)
        kda.attn_weights(pool, tables[turn], place, q_rot, lse, weights, err)
        at += T
        torch.cuda.synchronize()
        table, p0 = tables[turn].cpu().numpy(), place.tolist()
        kp, vp = f64(pool.k), f64(pool.v)
        if blocks:
            kp, vp = mo.unscaled(kp, f64(pool.k_scale), 16), mo.unscaled(vp, f64(pool.v_scale), 16)
        k_rot = mo.rotated(f64(k).reshape(-1, Hkv, d), axis_pos.flatten().tolist(), f64(cos_sin)).reshape(B, T, Hkv, d)
        for b in range(B):
            for h in range(Hkv):
                rows[b][h] += [(k_rot[b, i, h], f64(v)[b, i, h]) for i in range(T)]
                pl = np.arange(p0[b] + T)
                got_k, got_v = (x[table[b][pl // page], h, pl % page] for x in (kp, vp))
                want_k, want_v = (np.array([r[i] for r in rows[b][h]]) for i in (0, 1))
                assert got_k.shape == want_k.shape
                # Stored once (2^-8 or 2^-4), and once more for each cut or raised scale in 8 bits (subnormals only).
                half, tiny = (2.0 ** -4, 2.0 ** -6) if blocks else (2.0 ** -8, 0.0)
                for x, y in ((got_k, want_k), (got_v, want_v)):
                    assert (np.abs(x - y) <= half * np.abs(y) * 1.01 + tiny * 2.0 ** -6 + 1e-5).all()
                for i in range(T):
                    n = p0[b] + i + 1
                    for r in range(Hq // Hkv):
                        s = got_k[:n] @ f64(q_rot)[b, i, h * 2 + r] * d ** -0.5
                        e = np.exp(s - s.max())
                        assert np.abs(e @ got_v[:n] / e.sum() - f64(o)[b, i, h * 2 + r]).max() <= 2.0 ** -7 * np.abs(got_v[:n]).max()
        place += T
        if step in (9, 17):
            kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=dev)
            new_w, old_w = torch.empty_like(weights), weights
            n = place.tolist()
            kda.kv_evict(pool, tables[turn], place, weights, tables[1 - turn], place, new_w, kept, err, recent=recent)
            # Every token's weights over all rounds since it came: as many as query heads and rounds.
            assert place.tolist() == [keep] * B and min(n) > keep
            for b in range(B):
                for h in range(Hkv):
                    places = mo.keep_places(old_w[b, h].tolist(), n[b], keep, recent)
                    assert kept[b, h].tolist() == places
                    rows[b][h] = [rows[b][h][i] for i in places]
            weights, turn = new_w, 1 - turn
    assert err.item() == 0
