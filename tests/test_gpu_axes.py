"""Appends whose rotation has positions on several axes, on the GPU against the fp64 oracle."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from oracle import paged_oracle as po
from tests.pages_testutil import FORMS, Batch, check_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def with_axes(b, axes, seed=0, max_pos=500):
    """Positions of b's tokens on some axes, a rotation table for them, and an axis for each pair."""
    rng = np.random.default_rng(seed)
    dim = b.cos_sin.shape[1]
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    b.cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().to(b.device)
    b.at = torch.from_numpy(rng.integers(0, max_pos, (axes, b.N))).to(b.device)
    b.at[:, -1] = max_pos - 1
    return b


def reference(b, axis_of, pairs, skip=()):
    """(q, k pages, v pages) of the call; rows in `skip` are left out."""
    at, cs = b.at.T.cpu().numpy(), f64(b.cos_sin)
    at = np.where(np.isin(np.arange(b.N), skip)[:, None], 0, at)
    q = mo.rotated(f64(b.q), at, cs, axis_of, b.rot_start, pairs)
    k = mo.rotated(f64(b.k), at, cs, axis_of, b.rot_start, pairs)
    kp, vp = f64(b.k_pages), f64(b.v_pages)
    was = kp.copy(), None if vp is None else vp.copy()
    po.append(kp, vp, b.np_table(), b.pos.cpu().numpy(), b.counts, k, f64(b.v), None, None, 0, False, f64(b.k_scale),
              f64(b.v_scale))
    seq, tok = np.repeat(np.arange(b.B), b.counts), np.concatenate([np.arange(n) for n in b.counts])
    for r in skip:
        p = int(b.pos[seq[r]]) + tok[r]
        for x, x0 in zip((kp, vp), was):
            if x is not None:
                x[b.np_table()[seq[r]][p // b.page], :, p % b.page] = x0[b.np_table()[seq[r]][p // b.page], :, p % b.page]
    return q, kp, vp


def append(kda, b, axis_of, pairs=False, packed=True, q_out=None):
    q_out = torch.full_like(b.q, 7.0) if q_out is None else q_out
    kw = dict(cos_sin=b.cos_sin, rot_start=b.rot_start, rot_pairs=pairs, axis_of=axis_of)
    if packed:
        kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, q=b.q, q_out=q_out, axis_pos=b.at,
                      tok_start=b.tok_start, T=b.T, **kw)
    else:
        kda.kv_append(b.pool(kda), b.table, b.pos, b.dense(b.k), None if b.v is None else b.dense(b.v), b.err,
                      q=b.dense(b.q), q_out=b.dense(q_out), axis_pos=b.at.view(-1, b.B, b.T), **kw)
    torch.cuda.synchronize()
    return q_out


def check(b, ref, q_out):
    top = 2 * float(max(b.k.float().abs().max(), b.q.float().abs().max()))
    check_rows(q_out, ref[0], b.dt, top, "q")
    scale = 1.0 if b.k_scale is None else float(b.k_scale.min())
    check_rows(b.k_pages, ref[1], b.ct, top / scale, "k pages")
    if b.v_pages is not None:
        check_rows(b.v_pages, ref[2], b.ct, None, "v pages")


@pytest.mark.parametrize("form,packed,pairs", itertools.product(FORMS, [False, True], [False, True]))
def test_forms(kda, form, packed, pairs):
    counts = [3, 0, 1, 4] if packed else [3, 3, 3, 3]
    b = with_axes(Batch(form, Hq=8, Hkv=1 if form == "latent" else 2, page=16, pos=[0, 5, 15, 30], counts=counts,
                        seed=1), 3)
    half = b.cos_sin.shape[1] // 2
    axis_of = kda.rotation_axes([half - 2 * (half // 3), half // 3, half // 3], interleaved=packed)
    ref = reference(b, axis_of, pairs)
    check(b, ref, append(kda, b, axis_of, pairs, packed))
    assert b.err.item() == 0 and kda.last_variant() == "kv_append_axes"


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_any_axis_for_any_pair(kda, axes):
    """Random axes pair by pair, whole units of one axis, and one axis alone."""
    rng = np.random.default_rng(axes)
    for axis_of in (rng.integers(0, axes, 64).tolist(), np.repeat(np.arange(8) % axes, 8).tolist(), [axes - 1] * 64):
        b = with_axes(Batch("bf16_d128", Hq=6, Hkv=3, page=32, pos=[7, 100], counts=[40, 2], seed=axes), axes)
        ref = reference(b, axis_of, False)
        check(b, ref, append(kda, b, axis_of))


@pytest.mark.parametrize("start,dim,pairs", [(0, 64, False), (64, 64, True), (32, 16, False), (16, 96, True)])
def test_a_part_of_each_head(kda, start, dim, pairs):
    b = with_axes(Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[3, 9], counts=[5, 2], seed=7, rot_dim=dim), 2)
    b.rot_start = start
    axis_of = kda.rotation_axes([dim // 2 - dim // 4, dim // 4])
    ref = reference(b, axis_of, pairs)
    check(b, ref, append(kda, b, axis_of, pairs))


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "e4m3_d128", "latent"])
def test_equal_positions_are_the_plain_append(kda, form):
    mk = lambda: Batch(form, Hq=8, Hkv=1 if form == "latent" else 2, page=16, pos=[3, 20, 0], counts=[4, 1, 70], seed=3)  # noqa: E731
    a, b = mk(), mk()
    b.at = torch.cat([p + torch.arange(n, device=b.device) for p, n in zip([3, 20, 0], b.counts)]).expand(3, -1).contiguous()
    qa = torch.full_like(a.q, 7.0)
    kda.kv_append(a.pool(kda), a.table, a.pos, a.k, a.v, a.err, q=a.q, q_out=qa, cos_sin=a.cos_sin,
                  rot_start=a.rot_start, tok_start=a.tok_start, T=a.T)
    assert kda.last_variant() == "kv_append"
    half = b.cos_sin.shape[1] // 2
    qb = append(kda, b, kda.rotation_axes([half - 10, 5, 5], interleaved=True))
    assert torch.equal(qa, qb)
    for x, y in ((a.k_pages, b.k_pages), (a.v_pages, b.v_pages)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_places_past_the_rotation_table(kda):
    """What an evicted or very long cache needs: the place is no position."""
    b = with_axes(Batch("bf16_d64", Hq=2, Hkv=1, page=64, pos=[5000], counts=[3], seed=4), 1, max_pos=20)
    ref = reference(b, [0] * 32, False)
    check(b, ref, append(kda, b, None))
    assert b.err.item() == 0


def test_positions_outside_the_table_skip_their_token(kda):
    b = with_axes(Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[3, 9, 0], counts=[5, 2, 3], seed=8), 2, max_pos=50)
    b.at[1, 1], b.at[0, 5], b.at[1, 8] = 50, -1, 1 << 40
    axis_of = kda.rotation_axes([32, 32])
    ref = reference(b, axis_of, False, skip=(1, 5, 8))
    ref[0][[1, 5, 8]] = 7.0
    check(b, ref, append(kda, b, axis_of))
    assert b.err.item() == kda.DEV_ERR_POS


def test_places_below_zero_and_bad_pages(kda):
    b = with_axes(Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[3, 9], counts=[5, 12], seed=9), 2, max_pos=50)
    axis_of = kda.rotation_axes([32, 32])
    before = b.k_pages.clone()
    b.pos[0] = -2                     # two tokens without a place, three at 0, 1 and 2
    b.table[1, 1] = b.n_pages         # tokens 7 to 11 of the second sequence
    q_out = append(kda, b, axis_of)
    assert b.err.item() == kda.DEV_ERR_POS | kda.DEV_ERR_PAGE
    q = mo.rotated(f64(b.q), b.at.T.cpu().numpy(), f64(b.cos_sin), axis_of)
    gone = [0, 1] + list(range(12, 17))
    q[gone] = 7.0
    check_rows(q_out, q, b.dt, 2 * float(b.q.float().abs().max()), "q")
    k = mo.rotated(f64(b.k), b.at.T.cpu().numpy(), f64(b.cos_sin), axis_of)
    want = f64(before)
    for r, (s, p) in {2: (0, 0), 3: (0, 1), 4: (0, 2), **{5 + i: (1, 9 + i) for i in range(7)}}.items():
        want[b.np_table()[s][p // 16], :, p % 16] = k[r]
    check_rows(b.k_pages, want, b.ct, 2 * float(b.k.float().abs().max()), "k pages")


def test_a_long_prompt_in_place_on_another_stream(kda):
    """11000 tokens, which go past the caches, q rotated in place, on a stream of its own."""
    b = with_axes(Batch("bf16_d128", Hq=32, Hkv=8, page=64, pos=[10], counts=[11000], seed=5), 3, max_pos=4000)
    axis_of = kda.rotation_axes([20, 22, 22], interleaved=True)
    ref = reference(b, axis_of, False)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        append(kda, b, axis_of, q_out=b.q)
    check(b, ref, b.q)


def test_captured_call_replays(kda):
    """A captured append over changed tokens, positions and places gives the eager call's bits, replay after replay."""
    mk = lambda: with_axes(Batch("bf16_d128", Hq=8, Hkv=2, page=16, pos=[3, 20], counts=[4, 4], seed=6, extra_cols=2), 2)  # noqa: E731
    a, b = mk(), mk()
    axis_of = kda.rotation_axes([40, 24])
    for x in (a, b):
        x.table[x.table < 0] = 0
        x.q_out = torch.zeros_like(x.q)
        x.plan = kda.KvAppendPlan(x.pool(kda), x.table, x.pos, x.k, x.v, x.err, q=x.q, q_out=x.q_out,
                                  cos_sin=x.cos_sin, axis_pos=x.at, axis_of=axis_of, tok_start=x.tok_start, T=4)
    a.plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.plan()
    for step in range(4):
        for x in (a, b):
            g = torch.Generator(device=x.device).manual_seed(step)
            x.k.normal_(generator=g)
            x.q.normal_(generator=g)
            x.at.random_(0, 500, generator=g)
        a.plan()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.q_out, b.q_out) and torch.equal(a.k_pages, b.k_pages) and torch.equal(a.v_pages, b.v_pages)
    assert b.err.item() == 0
