"""How the paged attention's work is split: row blocks, tiles, workers' runs and pieces, and the loads that large pools
select."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.pages_testutil import FORMS, HALF_STEP, Batch, check_attend, f64

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
    scale = 192 ** -0.5
    ref = b.attend_ref(scale)
    o, lse = b.attend(kda, scale=scale)
    check_attend(o, lse, ref, b.dt, b.dk, 288)
    for _ in range(5):
        o2, lse2 = b.attend(kda, scale=scale)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert b.err.item() == 0


# ---------------------------------------------------------------- every token counts once

class Counted:
    """A cache that counts: queries are zero, so that every visible token weighs exactly 1, and token j's value is a one
    in column group(j).  With n visible tokens the sum is n, lse is log n, and column c of the output is the share of
    the visible tokens whose group is c.  All sums are whole numbers below 2^24, exact in 32 bits in any order and
    split.  Pages that hold no visible token, and the places around the sequences, hold NaN.

    seqs: (tokens cached, new tokens) of each sequence.  room: columns of the page table, at least those needed.
    pool_bytes: a pool of at least that size.
    """

    GROUP = 8  # neighbouring tokens that share a column

    def __init__(self, form, *, Hq, Hkv, page, seqs, T=None, window=0, room=0, pool_bytes=0, seed=0):
        self.dk, self.dv, self.dt, self.ct = FORMS[form]
        self.form, self.Hq, self.Hkv, self.page, self.seqs, self.window = form, Hq, Hkv, page, seqs, window
        self.T = T or max(max(n for _, n in seqs), 1)
        latent, rng, dev = form == "latent", np.random.default_rng(seed), "cuda"
        need = [max(0, -(-(p + n) // page)) if n else 0 for p, n in seqs]
        width = self.dk if latent else self.dk + self.dv
        per_page = Hkv * page * width * torch.empty(0, dtype=self.ct).element_size()
        n_pages = max(sum(need) + 2, pool_bytes // per_page + 1)
        self.n_pages, self.bytes = n_pages, n_pages * per_page
        ids = rng.permutation(n_pages)[:sum(need)]
        table, at = np.full((len(seqs), max(max(need), 1, room)), -1, np.int32), 0
        for b, m in enumerate(need):
            table[b, :m], at = ids[at:at + m], at + m
        self.table = torch.from_numpy(table).to(dev)
        self.pos = torch.tensor([p for p, _ in seqs], dtype=torch.int64, device=dev)
        self.starts = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
        self.tok_start = torch.from_numpy(self.starts.astype(np.int32)).to(dev)
        self.N = int(self.starts[-1])
        nan = torch.full((), float("nan"), device=dev).to(self.ct)

        def pages(w):
            x = torch.empty((n_pages, Hkv, page, w), dtype=self.ct, device=dev)
            (x.view(torch.uint8) if x.element_size() == 1 else x).fill_(
                nan.view(torch.uint8).item() if x.element_size() == 1 else float("nan"))
            return x

        self.k, self.v = pages(self.dk), None if latent else pages(self.dv)
        gen = torch.Generator(device=dev).manual_seed(seed)
        for b, (p0, n) in enumerate(seqs):
            lo, hi = self.visible(p0, p0 + n - 1)[0] if not window else max(0, p0 + 1 - window), p0 + n
            if n == 0 or hi <= 0:
                continue
            j = torch.arange(lo, hi, device=dev)
            pg, sl = self.table[b].long()[j // page], j % page
            key = torch.randn((len(j), Hkv, self.dk), device=dev, generator=gen).to(self.ct)
            one = torch.zeros((len(j), Hkv, self.dv), device=dev)
            one[torch.arange(len(j), device=dev), :, torch.from_numpy(self.column(j.cpu().numpy())).to(dev)] = 1.0
            one = one.to(self.ct)
            if latent:
                key[..., :self.dv] = one
            for x, y in ((self.k, key), (self.v, None if latent else one)):
                if x is not None:
                    bits = x.element_size() == 1
                    (x.view(torch.uint8) if bits else x)[pg, :, sl] = y.view(torch.uint8) if bits else y
        scale = torch.ones(Hkv, device=dev) if self.ct == torch.float8_e4m3fn else None
        self.scales = dict(k_scale=scale, v_scale=scale)

    def column(self, j):
        return (j // self.GROUP * 37 + j // (self.GROUP * self.dv)) % self.dv

    def visible(self, p0, p):
        return (max(0, p + 1 - self.window) if self.window else 0), p + 1

    def check(self, kda, what=""):
        pool = kda.PagePool.from_tensors(self.k, self.v, dv=self.dv, **self.scales)
        q = torch.zeros((self.N, self.Hq, self.dk), dtype=self.dt, device="cuda")
        o = torch.full((self.N, self.Hq, self.dv), 7.0, dtype=self.dt, device="cuda")
        lse = torch.empty((self.N, self.Hq), device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = kda.attn_workspace(pool, self.table, Hq=self.Hq, T=self.T)
        kda.attn_decode(pool, self.table, self.pos, q, o, ws, err, lse=lse, scale=1.0, window=self.window,
                        tok_start=self.tok_start, T=self.T)
        torch.cuda.synchronize()
        assert err.item() == 0, what
        o, lse = f64(o), f64(lse)
        for b, (p0, n) in enumerate(self.seqs):
            for i in range(n):
                lo, hi = self.visible(p0, p0 + i)
                r, seen = self.starts[b] + i, max(0, hi - lo)
                if seen == 0:
                    assert (o[r] == 0).all() and np.isneginf(lse[r]).all(), f"{what}: sequence {b}, token {i} sees nothing"
                    continue
                # The logarithm (2^-23 of it), its product with a rounded ln 2 (two halves of that): a token more or
                # less moves lse by 1 / n, which is more than this bound for n up to 170000.
                off = np.abs(lse[r] - np.log(seen)).max()
                assert off <= 4 * 2.0 ** -23 * max(np.log(seen), 1.0), \
                    f"{what}: sequence {b}, token {i}: {np.exp(lse[r]).round(2)} tokens counted of {seen}"
                want = np.bincount(self.column(np.arange(lo, hi)), minlength=self.dv) / seen
                # 1 / n, its product with the count, and the result's own type: half a step each.
                tol = want * (HALF_STEP[self.dt] + 4 * 2.0 ** -24)
                bad = np.abs(o[r] - want) > tol
                assert not bad.any(), f"{what}: sequence {b}, token {i}: columns {np.flatnonzero(bad.any(0))[:8]}, " \
                                      f"{(o[r].max(0) * seen).round(2)[bad.any(0)][:8]} for {(want * seen)[bad.any(0)][:8]}"


def ragged(B, T, seed, lengths=(-1, 0, 31, 40, 127, 300, 1300), p=(.05, .15, .2, .2, .1, .2, .1)):
    rng = np.random.default_rng(seed)
    return list(zip(rng.choice(lengths, B, p=p).tolist(), rng.integers(0, T + 1, B).tolist()))


GROUPED = [f for f in FORMS if f != "latent"]


@pytest.mark.parametrize("form", GROUPED)
@pytest.mark.parametrize("G,T", [(2, 1), (4, 4), (6, 5), (8, 8)])
def test_long_grouped_sequences_count_every_token(kda, form, G, T):
    """16, 32 and 64 rows to a workgroup (32 at most in fp32): one sequence over the whole chip, and a few."""
    for seqs in ([(20000, T)], [(131071 - T, T)] if T == 1 else [(9001, T)], [(6000, T), (100, 1), (2500, T), (-1, 1), (0, T)]):
        Counted(form, Hq=2 * G, Hkv=2, page=64, seqs=seqs, T=T, seed=61).check(kda, f"{form} {seqs}")


@pytest.mark.parametrize("hq,T,room", [(8, 2, 0), (16, 1, 4096), (32, 1, 4096), (16, 4, 4096), (32, 4, 8192), (33, 16, 2048)])
def test_long_latent_sequences_count_every_token(kda, hq, T, room):
    """Blocks of 16 to 128 rows (a wide table brings large ones)."""
    for seqs in ([(20000, T)], [(60001, T)], [(6000, T), (100, 1), (2500, T), (-1, 1), (0, T)]):
        Counted("latent", Hq=hq, Hkv=1, page=64, seqs=seqs, T=T, room=room, seed=62).check(kda, f"{hq} x {T} {seqs}")


@pytest.mark.parametrize("form", GROUPED)
@pytest.mark.parametrize("G,T,B", [(2, 2, 60), (2, 8, 100), (8, 4, 60), (8, 8, 90), (16, 8, 40), (1, 1, 600)])
@pytest.mark.parametrize("window", [0, 150])
def test_grouped_runs_over_several_sequences_count_every_token(kda, form, G, T, B, window):
    """More places in the list of tiles than workers: a worker's run ends one sequence, holds others and begins one."""
    Counted(form, Hq=8 * G, Hkv=8, page=32, seqs=ragged(B, T, B + T), T=T, window=window, seed=63).check(kda, form)


@pytest.mark.parametrize("hq,T,B", [(16, 1, 300), (32, 1, 200), (32, 4, 60), (64, 3, 70), (8, 8, 150)])
@pytest.mark.parametrize("window", [0, 150])
def test_latent_runs_over_several_sequences_count_every_token(kda, hq, T, B, window):
    Counted("latent", Hq=hq, Hkv=1, page=32, seqs=ragged(B, T, B + T), T=T, window=window, seed=64).check(kda)


@pytest.mark.parametrize("form", GROUPED)
@pytest.mark.parametrize("G,T", [(2, 4), (8, 4), (8, 8)])
def test_large_pools_count_every_token(kda, form, G, T):
    """Pools past 256 MB are read with loads of their own: few sequences, many, and a window."""
    big = dict(pool_bytes=(256 << 20) + (1 << 20), Hq=2 * G, Hkv=2, T=T, seed=65)
    c = Counted(form, page=64, seqs=[(5000, T), (-2, T), (130, 1)], **big)
    assert c.bytes > 256 << 20
    c.check(kda, form)
    Counted(form, page=128, seqs=ragged(200, T, 7), **big).check(kda, form)
    Counted(form, page=16, seqs=ragged(70, T, 8), window=40, **big).check(kda, form)


# ---------------------------------------------------------------- uneven batches against the oracle

@pytest.mark.parametrize("form", GROUPED)
@pytest.mark.parametrize("G,T,B", [(2, 2, 60), (4, 3, 80), (8, 4, 60), (12, 5, 45)])
def test_grouped_batches_of_uneven_sequences(kda, form, G, T, B):
    """Random queries, keys and values where test_grouped_runs_over_several_sequences counts; a refused page too."""
    seqs = ragged(B, T, 3 * B + T)
    b = Batch(form, Hq=4 * G, Hkv=4, page=32, pos=[p for p, _ in seqs], counts=[n for _, n in seqs], seed=66)
    for window in (33, 0):
        ref = b.attend_ref(window=window)
        o, lse = b.attend(kda, window=window)
        assert b.err.item() == 0
        check_attend(o, lse, ref, b.dt, b.dk, 1310, f"{form}, window {window}")
        o2, lse2 = b.attend(kda, window=window)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    starts = np.concatenate([[0], np.cumsum(b.counts)])
    long = [s for s, (p, n) in enumerate(seqs) if p == 1300 and n > 0]
    short = [s for s, (p, n) in enumerate(seqs) if p == 40 and n > 0]
    b.table[long[0], 17], b.table[short[0], 0] = b.n_pages, -5
    o, lse = b.attend(kda)
    assert b.err.item() == 32
    bad = [r for s in (long[0], short[0]) for r in range(starts[s], starts[s + 1])]
    rows = [r for r in range(b.N) if r not in bad]
    assert (o[bad] == 7).all() and (lse[bad] == 7).all()
    check_attend(o[rows], lse[rows], tuple(x[rows] for x in ref), b.dt, b.dk, 1310, f"{form}, two refused")


# ---------------------------------------------------------------- appends past the caches

@pytest.mark.parametrize("form", FORMS)
def test_large_appends_equal_small_ones(kda, form):
    """Above 256 MB an append goes past the caches: bit for bit what the same tokens leave in smaller calls."""
    dk, dv, dt, ct = FORMS[form]
    latent, Hq, Hkv, page = form == "latent", 8, 1 if form == "latent" else 2, 64
    e_in, e_c = (torch.empty(0, dtype=x).element_size() for x in (dt, ct))
    units = (Hq * dk + Hkv * (dk if latent else dk + dv)) // 16
    N = (256 << 20) // (units * 16 * (e_in + e_c)) + 777
    gen = torch.Generator(device="cuda").manual_seed(67)
    q, k, v = (torch.randn((N, h, w), device="cuda", generator=gen).to(dt) for h, w in ((Hq, dk), (Hkv, dk), (Hkv, dv)))
    v = None if latent else v
    first, dim = (dv, dk - dv) if latent else (0, dk)
    inv = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    ang = torch.arange(N + 5, device="cuda", dtype=torch.float64)[:, None] * inv
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
    n_pages = -(-(N + 5) // page)
    table = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)[None]
    scale = torch.tensor([0.013, 0.02], device="cuda") if ct == torch.float8_e4m3fn else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for step in (N, -(-N // 5)):
        pages = [None if w is None else torch.zeros((n_pages, Hkv, page, w), dtype=ct, device="cuda")
                 for w in (dk, None if latent else dv)]
        pool = kda.PagePool.from_tensors(*pages, dv=dv, k_scale=scale, v_scale=scale)
        q_out = torch.full_like(q, 7.0)
        for r in range(0, N, step):
            rows = slice(r, min(r + step, N))
            kda.kv_append(pool, table, torch.tensor([5 + r], device="cuda"), k[None, rows], None if latent else v[None, rows],
                          err, q=q[None, rows], q_out=q_out[None, rows], cos_sin=cos_sin, rot_start=first)
        torch.cuda.synchronize()
        got.append([x.view(torch.uint8) for x in (*pages, q_out) if x is not None])
    assert err.item() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)
