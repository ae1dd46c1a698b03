"""Sums of attention weights over the paged cache, on the GPU against the fp64 oracle."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from oracle import paged_oracle as po
from tests.blocks_testutil import BlockBatch
from tests.pages_testutil import FORMS, Batch, f64

pytestmark = pytest.mark.gpu

GROUPED = [f for f in FORMS if f != "latent"]


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def batch(form, **kw):
    return BlockBatch(int(form.split("_d")[1]), 16, **kw) if form.startswith("blocks") else Batch(form, **kw)


def key_values(b):
    if isinstance(b, BlockBatch):
        return b.values()[0]
    k = f64(b.k_pages)
    return k if b.k_scale is None else k * f64(b.k_scale)[:, None, None]


def prepared(b, scale=None, window=0, seed=0):
    """lse (fp32, of the oracle) and sums so far, with 7 behind the places of the table."""
    scale = b.dk ** -0.5 if scale is None else scale
    k = key_values(b)
    _, lse, _, _ = po.attend(k, k, b.np_table(), b.pos.cpu().numpy(), b.counts, f64(b.q), scale, window)
    b.lse = torch.from_numpy(lse).float().to(b.device)
    g = torch.Generator(b.device).manual_seed(seed)
    b.w = torch.rand((b.B, b.Hkv, b.table.shape[1] * b.page + 5), device=b.device, generator=g)
    return b


def run(kda, b, scale=None, window=0, packed=True, q=None):
    q = b.q if q is None else q
    if packed:
        kda.attn_weights(b.pool(kda), b.table, b.pos, q, b.lse, b.w, b.err, scale=scale, window=window,
                         tok_start=b.tok_start, T=b.T)
    else:
        kda.attn_weights(b.pool(kda), b.table, b.pos, b.dense(q), b.dense(b.lse), b.w, b.err, scale=scale, window=window)
    torch.cuda.synchronize()
    assert kda.last_variant() == "attn_weights"


def check(b, before, scale=None, window=0):
    """Against the oracle, from the roundings made.

    A score: a sum of dk products and dk additions, times the scale, log2 e and an 8-bit scale, at most
    ds = (2 dk + 4) 2^-24 of its terms' sum; lse: the product with log2 e, 2^-23 of it; their difference, 2^-24 of the
    larger.  All move e^x by the factor e^(+-d), d < 0.1: at most 2 d.  The exponential adds 2^-22, the sum of R terms
    R 2^-24, and adding the sum so far 2^-24 of the result.
    """
    scale = b.dk ** -0.5 if scale is None else scale
    pos = b.pos.cpu().numpy()
    want, added, spread = mo.weigh(key_values(b), b.np_table(), pos, b.counts, f64(b.q), f64(b.lse), f64(before), scale, window)
    top = np.abs(f64(b.lse)[np.isfinite(f64(b.lse))]).max(initial=0.0)
    d = (2 * b.dk + 4) * 2.0 ** -24 * spread + 2.0 ** -22 * (top + spread)
    tol = (2 * d + 2.0 ** -22 + (b.T * b.Hq // b.Hkv + 8) * 2.0 ** -24) * added + 2.0 ** -23 * np.abs(want)
    g = f64(b.w)
    off = ~(np.abs(g - want) <= tol)
    assert not off.any(), f"{off.sum()} of {off.size} off, worst {np.abs(g - want)[off].max()} for {np.abs(want[off]).max()}"
    untouched = (added == 0) & (want == f64(before))
    assert np.array_equal(g[untouched], f64(before)[untouched])


@pytest.mark.parametrize("form,packed", itertools.product(GROUPED + ["blocks_d64", "blocks_d128"], [False, True]))
def test_forms(kda, form, packed):
    counts = [3, 0, 1, 4] if packed else [2, 2, 2, 2]
    b = prepared(batch(form, Hq=8, Hkv=2, page=16, pos=[0, 5, 131, 300], counts=counts, seed=1, extra_cols=1))
    before = b.w.clone()
    run(kda, b, packed=packed)
    check(b, before)
    assert b.err.item() == 0


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (16, 1, 1), (24, 2, 2), (64, 4, 4), (7, 7, 3), (8, 2, 33), (12, 1, 128)])
@pytest.mark.parametrize("window", [0, 5, 100])
@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64"])
def test_rows_and_windows(kda, form, hq, hkv, T, window):
    """From one row to more than the registers hold; windows shorter and longer than the new tokens."""
    b = prepared(batch(form, Hq=hq, Hkv=hkv, page=32, pos=[0, 63, 400], counts=[T, max(T - 1, 1), T], seed=2), window=window)
    before = b.w.clone()
    run(kda, b, window=window)
    check(b, before, window=window)


@pytest.mark.parametrize("hq,hkv,T", [(8, 1, 5), (4, 2, 40), (8, 2, 70), (16, 1, 128)])
@pytest.mark.parametrize("form", GROUPED + ["blocks_d64", "blocks_d128"])
def test_many_rows(kda, form, hq, hkv, T):
    """More rows than a wave holds, in every form: tiles past the ring of sums, sequences of one tile, of a few, of none."""
    counts = [T, 0, T - 1, 1, T]
    b = prepared(batch(form, Hq=hq, Hkv=hkv, page=64, pos=[0, 9, 700, 1290, 31], counts=counts, seed=3), window=900)
    before = b.w.clone()
    run(kda, b, window=900)
    check(b, before, window=900)
    assert b.err.item() == 0
    again = b.w.clone()
    b.w.copy_(before)
    run(kda, b, window=900)
    assert torch.equal(b.w, again)


def test_two_calls_add_up(kda):
    b = prepared(batch("bf16_d64", Hq=4, Hkv=2, page=16, pos=[40, 9], counts=[1, 1], seed=3, extra_cols=1))
    b.table[b.table < 0] = 0
    before = b.w.clone()
    run(kda, b)
    check(b, before)
    b.pos += 1
    b.k_pages.normal_()
    first = b.w.clone()
    w = b.w
    prepared(b)
    b.w = w
    run(kda, b)
    check(b, first)


def test_nan_so_far_counts_only_where_it_is(kda):
    """A new token's sum begins at zero whatever was there; other tokens' sums are their own."""
    b = prepared(batch("bf16_d64", Hq=4, Hkv=2, page=16, pos=[40], counts=[3], seed=4))
    b.w[0, :, 40:] = float("nan")
    b.w[0, 1, 7] = float("inf")
    before = b.w.clone()
    run(kda, b)
    assert torch.isfinite(b.w[0, 0, :43]).all() and torch.isinf(b.w[0, 1, 7]) and torch.isnan(b.w[0, :, 43:]).all()
    before[0, :, 40:], before[0, 1, 7], b.w[0, 1, 7], b.w[0, :, 43:] = 0, 0, 0, 0
    want, added, _ = mo.weigh(key_values(b), b.np_table(), [40], [3], f64(b.q), f64(b.lse), f64(before), 0.125)
    want[0, 1, 7] = 0
    assert np.allclose(f64(b.w), want, rtol=1e-5, atol=1e-9)


def test_what_no_row_sees_does_not_matter(kda):
    """Keys of NaN past the end and before the window, rows that see nothing, and unread table entries."""
    b = prepared(batch("bf16_d128", Hq=4, Hkv=2, page=64, pos=[130, 0], counts=[2, 4], seed=5, extra_cols=1), window=40)
    b.pos[1] = -3
    prepared(b, window=40)
    before = b.w.clone()
    seen = np.zeros((b.n_pages, 64), bool)
    for s, (lo, hi) in enumerate(((91, 132), (0, 1))):
        for j in range(lo, hi):
            seen[b.np_table()[s][j // 64], j % 64] = True
    clean = b.k_pages.clone()
    b.k_pages[torch.from_numpy(~seen).to(b.device)[:, None, :, None].expand(b.k_pages.shape)] = float("nan")
    assert torch.isneginf(b.lse[2:5]).all()
    run(kda, b, window=40)
    b.k_pages.copy_(clean)
    check(b, before, window=40)
    assert b.err.item() == 0


def test_keys_that_are_infinite_for_rows_that_see_them(kda):
    """A key that makes a score -inf weighs nothing; one that only later rows see leaves the tokens of others alone."""
    b = batch("bf16_d64", Hq=2, Hkv=1, page=16, pos=[20], counts=[3], seed=6)
    b.q.abs_()
    b.k_pages[b.np_table()[0][0], :, 5] = float("-inf")
    prepared(b)
    assert torch.isfinite(b.lse).all()
    before = b.w.clone()
    run(kda, b)
    assert (b.w[0, 0, 5] == before[0, 0, 5]).item()
    assert torch.isfinite(b.w).all()


@pytest.mark.parametrize("B,tokens", [(1, 40000), (24, 2000), (200, 90)])
def test_splits(kda, B, tokens):
    """Sums over all tokens: every visible token counts once, however the work is split."""
    b = batch("blocks_d128", Hq=4, Hkv=2, page=64, pos=[max(0, tokens - 7 * i) for i in range(B)], counts=[1] * B, seed=7)
    o = torch.empty((b.N, 4, 128), dtype=b.dt, device=b.device)
    b.lse = torch.empty((b.N, 4), device=b.device)
    pool = b.pool(kda)
    ws = kda.attn_workspace(pool, b.table, Hq=4, T=1)
    kda.attn_decode(pool, b.table, b.pos, b.q, o, ws, b.err, lse=b.lse, tok_start=b.tok_start, T=1)
    b.w = torch.zeros((B, 2, b.table.shape[1] * b.page), device=b.device)
    run(kda, b)
    assert (b.w.double().sum(-1) - 2).abs().max() < 1e-4   # two query heads to a kv head, weights that sum to one
    j = torch.arange(b.w.shape[-1], device=b.device)
    assert ((b.w > 0) == (j <= b.pos[:, None])[:, None]).all()
    again = b.w.clone()
    b.w.zero_()
    run(kda, b)
    assert torch.equal(b.w, again)


@pytest.mark.parametrize("form", ["bf16_d128", "blocks_d64"])
@pytest.mark.parametrize("B,tokens,T", [(1, 20000, 64), (20, 1500, 33), (150, 80, 17)])
def test_splits_of_many_rows(kda, form, B, tokens, T):
    b = batch(form, Hq=8, Hkv=2, page=64, pos=[max(0, tokens - 7 * i) for i in range(B)], counts=[T] * B, seed=8)
    pool, q = b.pool(kda), b.dense(b.q)
    ws, lse = kda.attn_workspace(pool, b.table, Hq=8, T=16), []
    for t in range(0, T, 16):  # the attention takes 16 tokens of a sequence at most
        part = q[:, t:t + 16].contiguous()
        lse.append(torch.empty(part.shape[:3], device=b.device))
        kda.attn_decode(pool, b.table, b.pos + t, part, torch.empty_like(part), ws, b.err, lse=lse[-1])
    b.lse = torch.cat(lse, 1).flatten(0, 1)
    b.w = torch.zeros((B, 2, b.table.shape[1] * b.page), device=b.device)
    run(kda, b)
    # Four query heads to a kv head and T rows of each, weights that sum to one.  Each comes from two sums of dk
    # products in fp32, whose orders differ: scores of up to about 8 times 2 dk 2^-24 twice.
    assert (b.w.double().sum(-1) - 4 * T).abs().max() < 4 * T * 2 * 8 * 2 * b.dk * 2.0 ** -24
    j = torch.arange(b.w.shape[-1], device=b.device)
    assert ((b.w > 0) == (j < b.pos[:, None] + T)[:, None]).all()


def test_strided_queries_and_another_stream(kda):
    b = prepared(batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[40, 9], counts=[2, 2], seed=8))
    before = b.w.clone()
    wide = torch.randn((b.N, 8, 128), device=b.device).bfloat16()
    wide[:, :4] = b.q
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        run(kda, b, q=wide[:, :4])
    check(b, before)


def test_refusals(kda):
    """A range that does not fit and a position past the table skip the sequence, a bad page its tokens."""
    b = prepared(batch("bf16_d64", Hq=2, Hkv=1, page=16, pos=[40, 20, 50, 9], counts=[1, 1, 1, 1], seed=9))
    before = b.w.clone()
    b.pos[1] = 64                                      # the table has four pages
    b.table[2, 1] = b.n_pages
    run(kda, b)
    assert b.err.item() == kda.DEV_ERR_PAGE
    got = b.w.clone()
    assert torch.equal(got[1], before[1]) and torch.equal(got[2, :, 16:32], before[2, :, 16:32])
    b.table[2, 1] = 0
    b.pos[1] = 20
    b.w.copy_(before)
    run(kda, b)
    assert torch.equal(got[[0, 3]], b.w[[0, 3]]) and torch.equal(got[2, :, :16], b.w[2, :, :16])
    assert torch.equal(got[2, :, 32:], b.w[2, :, 32:])
    b.err.zero_()
    b.w.copy_(before)
    b.tok_start[1] = 3                                 # rows 0 .. 2 of at most one, then backwards
    run(kda, b)
    assert b.err.item() == kda.DEV_ERR_TOKENS
    assert torch.equal(b.w[:2], before[:2]) and torch.equal(b.w[2:, :, 32:], torch.cat([got[2:3], got[3:]])[:, :, 32:])


def test_captured_call_replays(kda):
    mk = lambda: prepared(batch("bf16_d128", Hq=8, Hkv=2, page=16, pos=[3, 40], counts=[2, 2], seed=10))  # noqa: E731
    a, b = mk(), mk()
    for x in (a, b):
        x.plan = kda.AttnWeightsPlan(x.pool(kda), x.table, x.pos, x.q, x.lse, x.w, x.err, tok_start=x.tok_start, T=2)
    a.plan()
    b.plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.plan()
    for step in range(4):
        for x in (a, b):
            x.q.normal_(generator=torch.Generator(x.device).manual_seed(step))
        a.plan()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.w, b.w)
