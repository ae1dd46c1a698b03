"""e4m3 pages with scales by blocks of tokens, on the GPU: appends and attention against the fp64 oracle."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from tests.blocks_testutil import BlockBatch, check_stored
from tests.pages_testutil import check_attend, check_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def run_append(kda, b, *, packed=True, pairs=False, with_q=True, rotated=True, in_place=False, axis_pos=None, axis_of=None):
    q_out = None if not with_q else b.q if in_place else torch.full_like(b.q, 7.0)
    kw = dict(q=b.q, q_out=q_out) if with_q else {}
    if rotated:
        kw |= dict(cos_sin=b.cos_sin, rot_start=b.rot_start, rot_pairs=pairs, axis_pos=axis_pos, axis_of=axis_of)
    if packed:
        kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=b.T, **kw)
    else:
        kw = {n: b.dense(x) if n in ("q", "q_out") else x for n, x in kw.items()}
        kda.kv_append(b.pool(kda), b.table, b.pos, b.dense(b.k), b.dense(b.v), b.err, **kw)
    torch.cuda.synchronize()
    assert kda.last_variant() == "kv_append_blocks"
    return q_out


def append_and_check(kda, b, *, pairs=False, rotated=True, axis_pos=None, axis_of=None, **kw):
    q0, k0 = f64(b.q), f64(b.k)
    at = np.concatenate([int(p) + np.arange(n) for p, n in zip(b.pos.tolist(), b.counts)]) if axis_pos is None else \
        axis_pos.T.cpu().numpy()
    turn = lambda x: mo.rotated(x, at, f64(b.cos_sin), axis_of, b.rot_start, pairs) if rotated else x  # noqa: E731
    was = [x.clone() for x in (b.k_pages, b.k_scale, b.v_pages, b.v_scale)]
    pos = b.pos.cpu().numpy()
    q_out = run_append(kda, b, pairs=pairs, rotated=rotated, axis_pos=axis_pos, axis_of=axis_of, **kw)
    if q_out is not None:
        check_rows(q_out, turn(q0), b.dt, 2 * np.abs(q0).max() if q0.size else 1.0, "q")
    # Two fp32 products and their sum, each half a step of values up to 2 max |k|.
    err = 4 * 2.0 ** -24 * 2 * np.abs(k0[np.isfinite(k0)]).max(initial=0.0) if rotated else 0.0
    check_stored(b.k_pages, b.k_scale, was[0], was[1], b.np_table(), pos, b.counts, turn(k0), b.block, err, "k")
    check_stored(b.v_pages, b.v_scale, was[2], was[3], b.np_table(), pos, b.counts, f64(b.v), b.block, 0.0, "v")
    assert b.err.item() == 0


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("width,block,packed,pairs", itertools.product([64, 128], [16, 32, 64], [False, True], [False, True]))
def test_append_forms(kda, width, block, packed, pairs):
    counts = [3, 0, 1, 4] if packed else [3, 3, 3, 3]
    b = BlockBatch(width, block, Hq=8, Hkv=2, page=64, pos=[0, 5, 15, 62], counts=counts, seed=1)
    append_and_check(kda, b, packed=packed, pairs=pairs)


@pytest.mark.parametrize("hq,hkv,page,block", [(1, 1, 1024, 256), (5, 5, 32, 16), (7, 1, 64, 64), (24, 8, 256, 128),
                                               (64, 4, 16, 16), (3, 3, 512, 256)])
def test_append_heads_pages_and_blocks(kda, hq, hkv, page, block):
    b = BlockBatch(128, block, Hq=hq, Hkv=hkv, page=page, pos=[page - 1, 2 * page, 0, block - 3], counts=[2, 1, 70, 6],
                   seed=3)
    append_and_check(kda, b)


@pytest.mark.parametrize("n,block", [(15, 16), (17, 32), (64, 64), (65, 64), (100, 128), (300, 256), (1100, 256),
                                     (1500, 128)])
def test_append_prompts(kda, n, block):
    """Blocks cut by a prompt's beginning and end."""
    b = BlockBatch(64, block, Hq=4, Hkv=2, page=max(block, 64), pos=[0, 37], counts=[n, n // 2], seed=n)
    append_and_check(kda, b)


def test_append_many_sequences(kda):
    rng = np.random.default_rng(0)
    b = BlockBatch(64, 16, Hq=2, Hkv=1, page=16, pos=rng.integers(0, 60, 300), counts=rng.integers(0, 4, 300), seed=5)
    append_and_check(kda, b)


def test_append_without_rotation_or_queries(kda):
    b = BlockBatch(128, 32, Hq=4, Hkv=2, page=32, pos=[3, 31], counts=[5, 40], seed=6)
    append_and_check(kda, b, with_q=False, rotated=False)
    b = BlockBatch(128, 32, Hq=4, Hkv=2, page=32, pos=[3, 31], counts=[5, 40], seed=6)
    append_and_check(kda, b, with_q=False)


def test_append_rotates_in_place_with_axes(kda):
    b = BlockBatch(128, 64, Hq=6, Hkv=2, page=64, pos=[3, 60], counts=[90, 9], seed=7, max_pos=400)
    at = torch.randint(0, 400, (3, b.N), device=b.device, generator=torch.Generator(b.device).manual_seed(1))
    append_and_check(kda, b, in_place=True, axis_pos=at, axis_of=kda.rotation_axes([20, 22, 22], interleaved=True))


@pytest.mark.parametrize("size", [0.0, 1e-25, 2.0 ** -40, 1e-4, 300.0, 448.0, 450.0, 1e5, 3e38])
def test_append_of_any_size_and_what_it_does_to_a_begun_block(kda, size):
    b = BlockBatch(64, 16, Hq=2, Hkv=2, page=32, pos=[9, 16, 0], counts=[2, 3, 20], seed=8)
    b.k.mul_(0.2 * size).clamp_(-size, size)
    b.v.mul_(0.2 * size).clamp_(-size, size)
    b.v[4, 1, 3] = size
    append_and_check(kda, b, rotated=False, with_q=False)


def test_append_infinities_and_nan(kda):
    b = BlockBatch(64, 16, Hq=2, Hkv=2, page=32, pos=[9, 0], counts=[2, 20], seed=9)
    b.k[0, 0, 5], b.k[3, 1, 7], b.v[4, 0, 0], b.v[0, 1, 1] = np.inf, -np.inf, np.nan, np.nan
    b.v[10, 1] = np.inf
    append_and_check(kda, b, rotated=False, with_q=False)
    b.v.fill_(np.nan)
    append_and_check(kda, b, rotated=False, with_q=False)


def test_scales_that_are_no_powers_of_two(kda):
    b = BlockBatch(64, 32, Hq=2, Hkv=2, page=32, pos=[9, 31], counts=[2, 3], seed=10)
    b.k_scale.mul_(1.3)
    b.v_scale.mul_(0.7)
    was = [x.clone() for x in (b.k_pages, b.k_scale)]
    k0 = f64(b.k)
    run_append(kda, b, rotated=False, with_q=False)
    want, scales = f64(was[0]), f64(was[1])
    mo.append_blocks(want, scales, b.np_table(), [9, 31], b.counts, k0, 32)
    assert np.array_equal(f64(b.k_scale), scales)
    # The factor old / new and its product with a value are fp32: two roundings before that to e4m3.
    assert (np.abs(f64(b.k_pages) - want) <= (2.0 ** -4 + 2.0 ** -22) * np.abs(want) + 2.0 ** -10).all()


def test_one_call_or_many_give_the_same_values(kda):
    """Token by token the scales end as in one call; values are rounded once more where a scale grew."""
    mk = lambda: BlockBatch(128, 64, Hq=4, Hkv=2, page=64, pos=[0, 64], counts=[50, 50], seed=11)  # noqa: E731
    a, b = mk(), mk()
    run_append(kda, a, rotated=False, with_q=False)
    k, v = b.dense(b.k), b.dense(b.v)
    pool = b.pool(kda)
    for i in range(50):
        kda.kv_append(pool, b.table, b.pos, k[:, i:i + 1], v[:, i:i + 1], b.err)
        b.pos += 1
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    for x, y in ((a.k_pages, b.k_pages), (a.v_pages, b.v_pages)):
        d = (x.float() - y.float()).abs()
        # Equal but where subnormal (below 2^-6): there a second and later roundings add half a step of 2^-9 each.
        assert (d[x.float().abs() >= 2.0 ** -5] == 0).all() and d.max() <= 2.0 ** -8


@pytest.mark.parametrize("width,block,T", [(128, 16, 12400), (128, 256, 12400), (64, 32, 24700), (128, 64, 4)])
def test_large_calls_write_what_small_ones_do(kda, width, block, T):
    """Calls past the size of the caches, against the same sequences in calls of at most 4096 tokens: bit for bit."""
    dev, B, Hq, Hkv, page = torch.device("cuda"), max(1, 12400 // T), 32, 8, 256
    if T == 4:  # many sequences, as in a round of drafts; 5 calls of a part of them each
        page = 64
    g = torch.Generator(device=dev).manual_seed(block)
    per = -(-T // page)
    n_pages = B * per
    qkv = torch.randn(B * T, (Hq + 2 * Hkv) * width, generator=g, device=dev).bfloat16()
    q, k, v = (x.unflatten(1, (-1, width)) for x in qkv.split([Hq * width, Hkv * width, Hkv * width], 1))
    assert qkv.numel() // qkv.shape[1] * width * (6 * Hkv + 4 * Hq) > 256 << 20
    cos_sin = torch.randn(T, width, generator=g, device=dev)
    table = torch.arange(n_pages, dtype=torch.int32, device=dev).view(B, per)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    got = []
    for at_once in (B * T, 4096):
        side = lambda: (torch.zeros(n_pages, Hkv, page, width, device=dev).to(torch.float8_e4m3fn),  # noqa: E731
                        torch.full((n_pages, Hkv, page // block), 2.0 ** -64, device=dev))
        (kp, ks), (vp, vs) = side(), side()
        pool = kda.PagePool.from_tensors(kp, vp, k_scale=ks, v_scale=vs, scale_block=block)
        out = torch.empty(B * T, Hq, width, dtype=torch.bfloat16, device=dev)
        if B == 1:
            calls = [(0, B, x, min(x + at_once, T)) for x in range(0, T, at_once)]
        else:
            calls = [(b, min(b + at_once // T, B), 0, T) for b in range(0, B, at_once // T)]
        for b0, b1, t0, t1 in calls:
            rows, n = slice(b0 * T + t0, (b1 - 1) * T + t1), t1 - t0
            start = torch.arange(0, (b1 - b0) * n + 1, n, dtype=torch.int32, device=dev)
            pos = torch.full((b1 - b0,), t0, dtype=torch.int64, device=dev)
            kda.kv_append(pool, table[b0:b1], pos, k[rows], v[rows], err, q=q[rows], q_out=out[rows], cos_sin=cos_sin,
                          tok_start=start, T=n)
        torch.cuda.synchronize()
        got.append((out, kp.view(torch.uint8), ks, vp.view(torch.uint8), vs))
    assert err.item() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_rejected_drafts_are_written_over(kda):
    b = BlockBatch(64, 16, Hq=2, Hkv=1, page=16, pos=[5], counts=[6], seed=12, extra_cols=1)
    b.table[b.table < 0] = 0
    b.v[3:] *= 1000  # rejected, and they raise the block's scale
    append_and_check(kda, b, rotated=False, with_q=False)
    raised = b.v_scale.clone()
    b.pos += 3
    b.counts, b.N, b.T = [2], 2, 2
    b.k, b.v, b.q = b.k[:2] * 0.5, b.v[:2] * 0.5, b.q[:2]
    b.tok_start = torch.tensor([0, 2], dtype=torch.int32, device=b.device)
    append_and_check(kda, b, rotated=False, with_q=False)
    assert torch.equal(b.v_scale, raised)


def test_append_refusals(kda):
    """Places below 0, past the rotation table and past the page table, bad pages, and ranges that do not fit."""
    b = BlockBatch(64, 16, Hq=2, Hkv=2, page=32, pos=[0, 40, 60, 10, 3], counts=[4, 4, 6, 4, 2], seed=13, max_pos=62)
    b.pos[0] = -2
    b.table[3, 0] = -1                                     # the fourth sequence's page
    was = [x.clone() for x in (b.k_pages, b.k_scale, b.v_pages, b.v_scale)]
    k0, v0, q0 = f64(b.k), f64(b.v), f64(b.q)
    q_out = run_append(kda, b)
    assert b.err.item() == kda.DEV_ERR_POS | kda.DEV_ERR_PAGE
    served = {2: (0, 0), 3: (0, 1), **{4 + i: (1, 40 + i) for i in range(4)}, 8: (2, 60), 9: (2, 61), 18: (4, 3), 19: (4, 4)}
    rows = sorted(served)
    q = np.full_like(q0, 7.0)
    at = [served[r][1] for r in rows]
    q[rows] = mo.rotated(q0[rows], at, f64(b.cos_sin))
    check_rows(q_out, q, b.dt, 2 * np.abs(q0).max(), "q")
    pos, counts = [0, 40, 60, 10, 3], [2, 4, 2, 0, 2]
    err = 4 * 2.0 ** -24 * 2 * np.abs(k0).max()
    table = b.np_table()
    check_stored(b.k_pages, b.k_scale, was[0], was[1], table, pos, counts, mo.rotated(k0[rows], at, f64(b.cos_sin)), 16,
                 err, "k")
    check_stored(b.v_pages, b.v_scale, was[2], was[3], table, pos, counts, v0[rows], 16, 0.0, "v")


def test_append_ranges_that_do_not_fit(kda):
    b = BlockBatch(64, 16, Hq=2, Hkv=2, page=32, pos=[0, 4, 8, 3], counts=[4, 3, 6, 4], seed=14)
    was = [x.clone() for x in (b.k_pages, b.k_scale, b.v_pages, b.v_scale)]
    k0, v0 = f64(b.k), f64(b.v)
    b.tok_start[1] = 9       # rows 0 .. 8: more than T = 6; rows 9 .. 6: backwards
    run_append(kda, b, rotated=False, with_q=False)
    assert b.err.item() == kda.DEV_ERR_TOKENS
    for got, scale, x, xs, new in ((b.k_pages, b.k_scale, was[0], was[1], k0), (b.v_pages, b.v_scale, was[2], was[3], v0)):
        check_stored(got, scale, x, xs, b.np_table(), [0, 4, 8, 3], [0, 0, 6, 4], new[7:], 16, 0.0)


def test_overlapping_ranges_serve_every_sequence(kda):
    """Ranges overlap where one between them runs backwards; more blocks then than the rows alone would have."""
    T, B = 20, 9
    b = BlockBatch(64, 16, Hq=1, Hkv=1, page=32, pos=[7] * B, counts=[T] * B, seed=15)
    was = [x.clone() for x in (b.v_pages, b.v_scale)]
    b.k, b.v = b.k[:T].contiguous(), b.v[:T].contiguous()
    ts = torch.tensor([0, T] * (B // 2) + [0, T], dtype=torch.int32, device=b.device)  # 0..T, T..0, 0..T, ...
    kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, tok_start=ts, T=T)
    assert b.err.item() == kda.DEV_ERR_TOKENS
    counts = [T if i % 2 == 0 else 0 for i in range(B)]
    rows = np.concatenate([f64(b.v)] * (B // 2 + 1))
    check_stored(b.v_pages, b.v_scale, *was, b.np_table(), [7] * B, counts, rows, 16, 0.0)


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("width,block,packed", itertools.product([64, 128], [16, 32, 64], [False, True]))
def test_attend_forms(kda, width, block, packed):
    counts = [3, 0, 1, 4] if packed else [2, 2, 2, 2]
    b = BlockBatch(width, block, Hq=8, Hkv=2, page=64, pos=[0, 5, 131, 300], counts=counts, seed=21)
    o, lse = b.attend(kda, packed=packed)
    assert kda.last_variant() == "attn_decode_blocks"
    check_attend(o, lse, b.attend_ref(), b.dt, b.dk, 310)
    assert b.err.item() == 0


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (16, 1, 1), (24, 2, 2), (64, 4, 16), (7, 7, 3)])
@pytest.mark.parametrize("window", [0, 5, 100])
def test_attend_heads_and_windows(kda, hq, hkv, T, window):
    b = BlockBatch(128, 32, Hq=hq, Hkv=hkv, page=128, pos=[0, 63, 500], counts=[T, T, T], seed=22)
    o, lse = b.attend(kda, window=window)
    check_attend(o, lse, b.attend_ref(window=window), b.dt, b.dk, 520)


def test_attend_scales_of_many_sizes(kda):
    """Blocks a factor 2^24 apart: what counts is scale times value."""
    b = BlockBatch(128, 16, Hq=8, Hkv=2, page=32, pos=[200, 1000], counts=[1, 2], seed=23, exps=(-30, -6))
    b.k_scale.copy_(2.0 ** torch.randint(-14, -7, b.k_scale.shape, device=b.device).float())
    o, lse = b.attend(kda)
    check_attend(o, lse, b.attend_ref(), b.dt, b.dk, 1010)
    b.v_scale *= 1.37  # not powers of two: the product with the probability is rounded once more, by 2^-24
    o, lse = b.attend(kda)
    check_attend(o, lse, b.attend_ref(), b.dt, b.dk, 1030)


def test_attend_ignores_what_no_row_sees(kda):
    """Codes of NaN, scales of NaN and infinity in blocks past the end, before the window and in spare pages."""
    b = BlockBatch(64, 16, Hq=4, Hkv=2, page=64, pos=[130, 70], counts=[2, 1], seed=24, extra_cols=1)
    ref = b.attend_ref(window=40)
    for pages, scale in ((b.k_pages, b.k_scale), (b.v_pages, b.v_scale)):
        seen, blocks = np.zeros((b.n_pages, 64), bool), np.zeros((b.n_pages, 4), bool)
        for s, (p, n) in enumerate(((130, 2), (70, 1))):
            for j in range(p + 1 - 40, p + n):
                page = b.np_table()[s][j // 64]
                seen[page, j % 64] = blocks[page, j % 64 // 16] = True
        dark = torch.from_numpy(~seen).to(b.device)[:, None, :, None].expand(pages.shape)
        pages.view(torch.uint8)[dark] = 0x7f
        scale[torch.from_numpy(~blocks).to(b.device)[:, None].expand(scale.shape)] = float("nan")
    o, lse = b.attend(kda, window=40)
    check_attend(o, lse, ref, b.dt, b.dk, 140)


def test_attend_not_finite_where_only_some_rows_see_it(kda):
    b = BlockBatch(64, 16, Hq=4, Hkv=2, page=64, pos=[100], counts=[4], seed=25)
    ref = b.attend_ref()
    page = b.np_table()[0][102 // 64]
    b.v_pages.view(torch.uint8)[page, :, 102 % 64] = 0x7f   # NaN: seen by the third and fourth token only
    o, lse = b.attend(kda)
    assert torch.isnan(o[2:]).all() and not torch.isnan(o[:2]).any()
    check_attend(o[:2], lse[:2], [x[:2] for x in ref], b.dt, b.dk, 110)


@pytest.mark.parametrize("B,tokens", [(1, 40000), (24, 2000), (200, 90)])
def test_attend_splits(kda, B, tokens):
    """Long sequences cut over many workers, batches on both ways of splitting: against the same values in f32 pages."""
    b = BlockBatch(128, 64, Hq=4, Hkv=2, page=64, pos=[max(0, tokens - 7 * i) for i in range(B)], counts=[1] * B, seed=26)
    o, lse = b.attend(kda)
    k, v = b.values()
    kv = [torch.from_numpy(x).float().to(b.device) for x in (k, v)]
    pool = kda.PagePool.from_tensors(*kv)
    ws = kda.attn_workspace(pool, b.table, Hq=b.Hq, T=1)
    o32, lse32 = torch.empty(b.N, b.Hq, 128, device=b.device), torch.empty(b.N, b.Hq, device=b.device)
    kda.attn_decode(pool, b.table, b.pos, b.q.float(), o32, ws, b.err, lse=lse32, tok_start=b.tok_start, T=1)
    # Probabilities (2^-8, on average none) and the result are rounded to bf16; |o| <= max |v|.
    assert (lse - lse32).abs().max() <= 1e-4
    assert (o.float() - o32).abs().max() <= 2.0 ** -8 * (o32.abs().max() + kv[1].abs().max())
    assert b.err.item() == 0


def test_attend_bad_pages(kda):
    b = BlockBatch(64, 16, Hq=4, Hkv=2, page=16, pos=[40, 40], counts=[1, 1], seed=27)
    ref = b.attend_ref()
    b.table[0, 1] = b.n_pages + 5
    o, lse = b.attend(kda)
    assert b.err.item() == kda.DEV_ERR_PAGE and (o[0] == 7).all() and (lse[0] == 7).all()
    check_attend(o[1:], lse[1:], [x[1:] for x in ref], b.dt, b.dk, 41)


def test_append_then_attend(kda):
    """A prompt, then decode steps with drafts: the attention sees what the appends stored."""
    b = BlockBatch(128, 32, Hq=8, Hkv=2, page=64, pos=[0, 0, 0], counts=[100, 31, 7], seed=28, extra_cols=2)
    b.table[b.table < 0] = 0
    run_append(kda, b, with_q=False)
    b.pos += torch.tensor(b.counts, device=b.device)
    for step in range(3):
        counts = [1, 2, 4]
        b.counts, b.N, b.T = counts, 7, 4
        b.tok_start = torch.tensor([0, 1, 3, 7], dtype=torch.int32, device=b.device)
        g = torch.Generator(b.device).manual_seed(step)
        b.q, b.k, b.v = (torch.randn((7, h, 128), device=b.device, generator=g).bfloat16() for h in (8, 2, 2))
        b.k *= 2 ** step
        b.cos_sin = torch.cat([torch.ones(200, 64), torch.zeros(200, 64)], 1).to(b.device)
        append_and_check(kda, b)
        o, lse = b.attend(kda)
        check_attend(o, lse, b.attend_ref(), b.dt, b.dk, 120)
        b.pos += torch.tensor(counts, device=b.device)


def test_captured_round_replays(kda):
    """Append and attend captured together, positions moved on by the graph: every replay gives the eager round's bits."""
    mk = lambda: BlockBatch(128, 16, Hq=8, Hkv=2, page=16, pos=[3, 40], counts=[2, 2], seed=29, extra_cols=2, spare=6)  # noqa: E731
    a, b = mk(), mk()
    for x in (a, b):
        free = [i for i in range(x.n_pages) if i not in x.np_table()]
        x.table[x.table < 0] = torch.tensor(free[:int((x.table < 0).sum())], dtype=torch.int32, device=x.device)
        x.p = x.pool(kda)
        x.o, x.lse = torch.zeros_like(x.q), torch.zeros((x.N, 8), device=x.device)
        x.ws = kda.attn_workspace(x.p, x.table, Hq=8, T=2)
        x.ap = kda.KvAppendPlan(x.p, x.table, x.pos, x.k, x.v, x.err, tok_start=x.tok_start, T=2)
        x.at = kda.AttnDecodePlan(x.p, x.table, x.pos, x.q, x.o, x.ws, x.err, lse=x.lse, tok_start=x.tok_start, T=2)

    def one(x):
        x.ap()
        x.at()
        x.pos.add_(2)
    one(a)
    one(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(b)
    for step in range(4):
        for x in (a, b):
            g = torch.Generator(x.device).manual_seed(step)
            for t in (x.q, x.k, x.v):
                t.normal_(generator=g)
            x.k.mul_(3.0 ** step)
        one(a)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in ((a.o, b.o), (a.lse, b.lse), (a.k_scale, b.k_scale), (a.k_pages.view(torch.uint8), b.k_pages.view(torch.uint8)),
                     (a.v_pages.view(torch.uint8), b.v_pages.view(torch.uint8))):
            assert torch.equal(x, y)
    assert b.err.item() == 0
