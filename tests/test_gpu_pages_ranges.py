"""Token ranges of the paged attention calls: packed rows that belong to no sequence, before, between and behind the
sequences' own, and who gets which row."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests.pages_testutil import Batch, check_attend, check_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def served(starts, N, T):
    """(sequence, first row, tokens) of the ranges that fit the launch."""
    return [(b, r0, r1 - r0) for b, (r0, r1) in enumerate(zip(starts, starts[1:])) if 0 <= r0 <= r1 <= N and r1 - r0 <= T]


def run_ranges(kda, form, hq, hkv, starts, N, T, seed, pairs=False):
    """append and attend with these ranges: every sequence that fits is served, row for row, and nothing else is
    written.  Returns the error word."""
    B = len(starts) - 1
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 40, B)
    b = Batch(form, Hq=hq, Hkv=hkv, page=16, pos=pos, counts=[max(T, -(-N // B))] * B, seed=seed)
    q, k, v = (None if x is None else x[:N].contiguous() for x in (b.q, b.k, b.v))
    ts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    seqs, table, cs = served(starts, N, T), b.np_table(), f64(b.cos_sin)
    kp, vp, q_ref = f64(b.k_pages), f64(b.v_pages), np.zeros((N, hq, b.dk))
    before = [None if x is None else x.clone() for x in (b.k_pages, b.v_pages)]
    touched, owned = torch.zeros((b.n_pages, b.page), dtype=torch.bool), np.zeros(N, dtype=int)
    for s, r0, n in seqs:
        rows = slice(r0, r0 + n)
        q_ref[rows] = po.append(kp, vp, table[s:s + 1], pos[s:s + 1], [n], f64(k[rows]), None if v is None else f64(v[rows]),
                                f64(q[rows]), cs, b.rot_start, pairs, f64(b.k_scale), f64(b.v_scale))
        owned[rows] += 1
        for p in range(pos[s], pos[s] + n):
            touched[table[s][p // 16], p % 16] = True
    pool, q_out = b.pool(kda), torch.full_like(q, 7.0)
    kda.kv_append(pool, b.table, b.pos, k, v, b.err, q=q, q_out=q_out, cos_sin=b.cos_sin, rot_start=b.rot_start,
                  rot_pairs=pairs, tok_start=ts, T=T)
    torch.cuda.synchronize()
    top = 2 * float(max(k.float().abs().max(), q.float().abs().max()))
    scale = 1.0 if b.k_scale is None else float(b.k_scale.min())
    for x, x0, want, terms in ((b.k_pages, before[0], kp, top / scale), (b.v_pages, before[1], vp, None)):
        if x is None:
            continue
        at = touched.nonzero(as_tuple=True)
        new = x.float()[at[0], :, at[1]]
        check_rows(new, want[at[0], :, at[1]], x.dtype, terms, f"{form} {starts}: pages")
        same = (x.view(torch.uint8) == x0.view(torch.uint8)).view(b.n_pages, -1, b.page, x.shape[-1] * x.element_size())
        assert same.all(dim=(1, 3)).cpu()[~touched].all(), f"{form} {starts}: a place of no token was written"
    once = np.flatnonzero(owned == 1)
    check_rows(q_out[once], q_ref[once], b.dt, top, f"{form} {starts}: q")
    assert (q_out[np.flatnonzero(owned == 0)] == 7).all(), f"{form} {starts}: a row of no sequence was written"
    # The same ranges read back.
    o, lse = torch.full((N, hq, b.dv), 7.0, dtype=b.dt, device="cuda"), torch.full((N, hq), 7.0, device="cuda")
    ws = kda.attn_workspace(pool, b.table, Hq=hq, T=T)
    kda.attn_decode(pool, b.table, b.pos, q, o, ws, b.err, lse=lse, scale=b.dk ** -0.5, tok_start=ts, T=T)
    torch.cuda.synchronize()
    for s, r0, n in seqs:
        rows = [r for r in range(r0, r0 + n) if owned[r] == 1]
        if rows:
            ref = po.attend(f64(b.k_pages), f64(b.v_pages), table[s:s + 1], pos[s:s + 1], [n], f64(q[r0:r0 + n]),
                            b.dk ** -0.5, 0, f64(b.k_scale), f64(b.v_scale), b.dv)
            pick = [r - r0 for r in rows]
            check_attend(o[rows], lse[rows], tuple(x[pick] for x in ref), b.dt, b.dk, 64, f"{form} {starts}: sequence {s}")
    none = np.flatnonzero(owned == 0)
    assert (o[none] == 7).all() and (lse[none] == 7).all()
    return b.err.item()


@pytest.mark.parametrize("form,hq,hkv", [("bf16_d64", 2, 1), ("bf16_d64", 2, 2), ("f32_d64", 1, 1), ("e4m3_d128", 4, 2),
                                         ("latent", 1, 1), ("latent", 32, 1)])
@pytest.mark.parametrize("starts,N,T", [([1, 3], 3, 2), ([1, 3, 5], 5, 2), ([1, 2], 2, 1), ([5, 5, 8, 8, 12], 14, 4),
                                        ([70, 70, 70, 71, 74], 75, 4)])
def test_rows_before_the_first_sequence(kda, form, hq, hkv, starts, N, T):
    """A wave that begins in rows of no sequence still serves the rows that follow."""
    assert run_ranges(kda, form, hq, hkv, starts, N, T, seed=41) == 0


@pytest.mark.parametrize("form,hq,hkv", [("bf16_d64", 2, 2), ("f32_d64", 1, 1), ("e4m3_d128", 4, 2), ("latent", 16, 1)])
@pytest.mark.parametrize("starts,N,T", [([0, 3, 4, 4, 7, 25, 10, 13, 17, 17, 20], 20, 4), ([0, 1000, 1000, 6, 9], 9, 3),
                                        ([-2, 1, 3, 5], 5, 2), ([2, 0, 2, 4], 4, 2), ([0, 2, -1000, 4, 6], 6, 2),
                                        ([0, 9, 9, 12, 14], 14, 3)])
def test_a_bad_range_takes_nothing_from_the_others(kda, form, hq, hkv, starts, N, T):
    assert run_ranges(kda, form, hq, hkv, starts, N, T, seed=42) == 128


@pytest.mark.parametrize("form,hq,hkv", [("bf16_d64", 2, 1), ("latent", 2, 1)])
@pytest.mark.parametrize("at,to", [(63, 10 ** 6), (64, 10 ** 6), (63, -7), (1, 2 ** 31 - 1), (1, -2 ** 31), (129, 10 ** 6),
                                   (0, 10 ** 6), (100, 0)])
def test_a_bad_range_among_many_sequences(kda, form, hq, hkv, at, to):
    """One entry changed in a list of 130 sequences, idle ones among them."""
    counts = np.random.default_rng(1).integers(0, 4, 130)
    counts[[0, 62, 63, 64, 99, 100, 128, 129]] = 2
    starts = [0, *np.cumsum(counts).tolist()]
    N = starts[-1]
    starts[at] = to
    assert run_ranges(kda, form, hq, hkv, starts, N, 3, seed=43) == 128


@pytest.mark.parametrize("form,hq,hkv", [("bf16_d64", 2, 2), ("e4m3_d128", 2, 1), ("latent", 8, 1)])
@pytest.mark.parametrize("starts,N,T", [([0, 3, 1, 4], 4, 3), ([0, 4, 0, 4, 0, 4], 4, 4), ([1, 3, 2, 4, 3, 6], 7, 3)])
def test_ranges_that_overlap(kda, form, hq, hkv, starts, N, T):
    """Each sequence's tokens reach its own pages, also from a row that a second sequence's range holds."""
    assert run_ranges(kda, form, hq, hkv, starts, N, T, seed=44) == 128


def test_many_sequences_with_gaps(kda):
    """Sequences of one token among idle ones, with rows of no sequence in front and behind."""
    counts = np.random.default_rng(2).integers(0, 2, 300)
    starts = [9, *(9 + np.cumsum(counts)).tolist()]
    assert run_ranges(kda, "bf16_d64", 1, 1, starts, starts[-1] + 20, 1, seed=45) == 0


@pytest.mark.parametrize("at", [2, 255, 256, 257, 511, 512, 513, 598])
@pytest.mark.parametrize("back", [10 ** 6, 2])
def test_a_bad_range_among_hundreds(kda, at, back):
    """Lists that are read 256 ranges at a time, and the rest: one entry far off, or one that reaches back over the
    rows of sequences before (a sequence without tokens between them runs backwards)."""
    counts = np.random.default_rng(3).integers(0, 4, 600)
    counts[[at - 2, at - 1, at]] = 2, 0, 2
    starts = [0, *np.cumsum(counts).tolist()]
    starts[at] = starts[at] + back if back > 5 else starts[at] - back
    assert run_ranges(kda, "bf16_d64", 2, 1, starts, int(counts.sum()), 5, seed=46) == 128


@pytest.mark.parametrize("what,bit", [("page", 32), ("pos", 64)])
def test_errors_of_a_second_sequence_are_named(kda, what, bit):
    """A row's second sequence has its own position and pages, and its own errors."""
    b = Batch("bf16_d64", Hq=2, Hkv=1, page=16, pos=[4, 0, 9], counts=[3, 3, 3], seed=47)
    q, k, v = (x[:4].contiguous() for x in (b.q, b.k, b.v))
    if what == "page":
        b.table[2] = -1
    else:
        b.pos[2] = -3
    ts = torch.tensor([0, 3, 1, 3], dtype=torch.int32, device="cuda")      # sequence 2's rows are sequence 0's
    kp = f64(b.k_pages)
    po.append(kp, f64(b.v_pages), b.np_table()[:1], np.array([4]), [3], f64(k[:3]), f64(v[:3]), f64(q[:3]), f64(b.cos_sin))
    kda.kv_append(b.pool(kda), b.table, b.pos, k, v, b.err, q=q, q_out=torch.empty_like(q), cos_sin=b.cos_sin, tok_start=ts,
                  T=3)
    assert b.err.item() == 128 | bit
    check_rows(b.k_pages, kp, b.ct, 2 * float(k.float().abs().max()))


@pytest.mark.parametrize("form,hq,hkv", [("bf16_d64", 2, 1), ("latent", 1, 1)])
def test_rows_of_very_many_sequences(kda, form, hq, hkv):
    """Ranges forth and back over the same rows: each turn of a row's search goes on where the one before met a
    sequence."""
    assert run_ranges(kda, form, hq, hkv, [0, 2] * 1500 + [1, 3], 3, 2, seed=48) == 128
