"""The paged attention calls on the GPU against the fp64 oracle: forms, layouts, sizes, masks, refusals, streams, graphs,
and a run of the calls beside the recurrent ones."""

from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

import synth
from oracle import kda_oracle as ko
from tests.kda_testutil import assert_parity, dev_inputs, dev_tensor, say, token_slice
from tests.pages_testutil import FORMS, Batch, check_attend, check_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def heads(form, hq=8, hkv=2):
    return dict(Hq=hq, Hkv=1 if form == "latent" else hkv)


# ---------------------------------------------------------------- append

def run_append(kda, b, *, packed=True, pairs=False, with_q=True, rotated=True, in_place=False):
    q_out = None if not with_q else b.q if in_place else torch.full_like(b.q, 7.0)
    kw = dict(q=b.q, q_out=q_out) if with_q else {}
    if rotated:
        kw |= dict(cos_sin=b.cos_sin, rot_start=b.rot_start, rot_pairs=pairs)
    if packed:
        kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=b.T, **kw)
    else:
        kw = {n: b.dense(x) if n in ("q", "q_out") else x for n, x in kw.items()}
        kda.kv_append(b.pool(kda), b.table, b.pos, b.dense(b.k), None if b.v is None else b.dense(b.v), b.err, **kw)
    torch.cuda.synchronize()
    assert kda.last_variant() == "kv_append"
    return q_out


def check_append(b, ref, q_out):
    q_ref, k_ref, v_ref = ref
    top = 2 * float(max(b.k.float().abs().max(), b.q.float().abs().max())) if b.N else 1.0
    if q_out is not None:
        check_rows(q_out, q_ref, b.dt, top, "q")
    scale = 1.0 if b.k_scale is None else float(b.k_scale.min())
    check_rows(b.k_pages, k_ref, b.ct, top / scale, "k pages")
    if b.v_pages is not None:
        check_rows(b.v_pages, v_ref, b.ct, None, "v pages")


@pytest.mark.parametrize("form,packed,pairs", itertools.product(FORMS, [False, True], [False, True]))
def test_append_forms(kda, form, packed, pairs):
    counts = [3, 0, 1, 4] if packed else [3, 3, 3, 3]
    b = Batch(form, **heads(form), page=16, pos=[0, 5, 15, 30], counts=counts, seed=1)
    ref = b.append_ref(pairs)
    q_out = run_append(kda, b, packed=packed, pairs=pairs)
    check_append(b, ref, q_out)
    assert b.err.item() == 0


@pytest.mark.parametrize("form", FORMS)
def test_append_leaves_every_other_place_as_it_was(kda, form):
    b = Batch(form, **heads(form), page=16, pos=[7, 0], counts=[2, 17], seed=2)
    before = [None if x is None else x.clone() for x in (b.k_pages, b.v_pages)]
    run_append(kda, b)
    touched = torch.zeros((b.n_pages, b.page), dtype=torch.bool)
    table = b.np_table()
    for s, (p0, n) in enumerate(zip([7, 0], [2, 17])):
        for p in range(p0, p0 + n):
            touched[table[s][p // 16], p % 16] = True
    for x, y in zip(before, (b.k_pages, b.v_pages)):
        if x is not None:
            same = (x.view(torch.uint8) == y.view(torch.uint8)).view(b.n_pages, -1, b.page, x.shape[-1] * x.element_size())
            assert same.all(dim=(1, 3)).cpu()[~touched].all()


@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 1024), (5, 5, 32), (7, 1, 64), (24, 8, 256), (64, 4, 16)])
def test_append_heads_and_pages(kda, hq, hkv, page):
    b = Batch("bf16_d128", Hq=hq, Hkv=hkv, page=page, pos=[page - 1, 2 * page, 0], counts=[2, 1, 70], seed=3)
    ref = b.append_ref()
    check_append(b, ref, run_append(kda, b))


def test_append_prompt_and_many_sequences(kda):
    b = Batch("bf16_d64", Hq=4, Hkv=2, page=64, pos=[0], counts=[1500], seed=4)
    ref = b.append_ref()
    check_append(b, ref, run_append(kda, b, packed=False))
    rng = np.random.default_rng(0)
    b = Batch("e4m3_d64", Hq=2, Hkv=1, page=16, pos=rng.integers(0, 60, 300), counts=rng.integers(0, 4, 300), seed=5)
    ref = b.append_ref()
    check_append(b, ref, run_append(kda, b))


def test_append_without_rotation_or_queries(kda):
    b = Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[3], counts=[5], seed=6)
    _, k_ref, v_ref = b.append_ref(rotated=False, with_q=False)
    run_append(kda, b, with_q=False, rotated=False)
    assert np.array_equal(f64(b.k_pages), k_ref) and np.array_equal(f64(b.v_pages), v_ref)
    b = Batch("f32_d64", Hq=4, Hkv=2, page=16, pos=[3], counts=[5], seed=6)
    ref = b.append_ref(with_q=False)
    run_append(kda, b, with_q=False)
    check_append(b, ref, None)


@pytest.mark.parametrize("start,dim,pairs", [(0, 64, False), (64, 64, True), (32, 16, False), (16, 96, True)])
def test_append_rotates_a_part_of_each_head(kda, start, dim, pairs):
    b = Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[3, 9], counts=[5, 2], seed=7, rot_dim=dim)
    b.rot_start = start
    ref = b.append_ref(pairs)
    check_append(b, ref, run_append(kda, b, pairs=pairs))


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "latent"])
def test_append_in_place_and_from_slices(kda, form):
    """q rotated in place, and q, k, v as slices of one projection: the bits of the dense call."""
    b = Batch(form, **heads(form), page=16, pos=[3, 9], counts=[4, 4], seed=8)
    pages0 = [None if x is None else x.clone() for x in (b.k_pages, b.v_pages)]
    q_out = run_append(kda, b, packed=False)
    want = [None if x is None else x.clone() for x in (b.k_pages, b.v_pages)]
    for x, x0 in zip((b.k_pages, b.v_pages), pages0):
        if x is not None:
            x.copy_(x0)
    Hkv = b.k.shape[1]
    if b.latent:
        qkv = torch.cat([b.dense(b.q), b.dense(b.k)], 2)
        q, k, v = qkv[:, :, :b.Hq], qkv[:, :, b.Hq:], None
    else:
        qkv = torch.cat([b.dense(b.q), b.dense(b.k), b.dense(b.v)], 2)
        q, k, v = qkv[:, :, :b.Hq], qkv[:, :, b.Hq:b.Hq + Hkv], qkv[:, :, b.Hq + Hkv:]
    kda.kv_append(b.pool(kda), b.table, b.pos, k, v, b.err, q=q, q_out=q, cos_sin=b.cos_sin, rot_start=b.rot_start)
    assert torch.equal(q.reshape(q_out.shape), q_out) and torch.equal(k.reshape(b.k.shape), b.k)
    for x, y in zip((b.k_pages, b.v_pages), want):
        assert x is None or torch.equal(x, y)


def test_append_e4m3_range(kda):
    b = Batch("e4m3_d64", Hq=2, Hkv=2, page=16, pos=[0], counts=[6], seed=9, rot_dim=16)
    b.k[0], b.k[1], b.k[2] = 1e30, -1e30, float("inf")
    b.v[3], b.v[4], b.v[5] = float("nan"), 1e-6, float("-inf")
    b.rot_start = 0
    kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=6)   # not rotated
    page = b.np_table()[0][0]
    k, v = b.k_pages[page].float(), b.v_pages[page].float()
    assert (k[:, 0] == 448).all() and (k[:, 1] == -448).all() and (k[:, 2] == 448).all()
    assert v[:, 3].isnan().all() and (v[:, 4] == 0).all() and (v[:, 5] == -448).all()


@pytest.mark.parametrize("what,bit", [("page", 32), ("page_high", 32), ("table", 32), ("neg", 64), ("far", 64),
                                      ("backwards", 128), ("long", 128), ("past", 128)])
def test_append_refuses_on_the_device(kda, what, bit):
    """A bad token or sequence is named and left out; the others are appended."""
    b = Batch("bf16_d64", Hq=2, Hkv=2, page=16, pos=[14, 3, 20], counts=[4, 2, 3], seed=10, max_pos=64)
    T, keep = 4, {0, 1, 2}
    good = Batch("bf16_d64", Hq=2, Hkv=2, page=16, pos=[14, 3, 20], counts=[4, 2, 3], seed=10, max_pos=64)
    skipped = range(6, 9)                                # rows of sequence 2
    if what == "page":
        b.table[2, 1] = -7
    elif what == "page_high":
        b.table[2, 1] = b.n_pages
    elif what == "table":
        b.pos[2] = 16 * b.table.shape[1]
        b.cos_sin = b.cos_sin.repeat(100, 1)
    elif what == "neg":
        b.pos[2] = -3
    elif what == "far":
        b.cos_sin = b.cos_sin[:20].contiguous()
    elif what == "backwards":
        b.tok_start[3] = 2
    elif what == "long":
        T, skipped = 3, range(0, 4)
    else:
        b.tok_start[3] = 10
    q_ref, k_ref, v_ref = good.append_ref()
    q_out = torch.full_like(b.q, 7.0)
    kda.kv_append(b.pool(kda), b.table, b.pos, b.k, b.v, b.err, q=b.q, q_out=q_out, cos_sin=b.cos_sin,
                  tok_start=b.tok_start, T=T)
    torch.cuda.synchronize()
    assert b.err.item() == bit
    rows = [r for r in range(9) if r not in skipped]
    top = 2 * float(b.q.float().abs().max())
    check_rows(q_out[rows], q_ref[rows], b.dt, top)
    assert (q_out[list(skipped)] == 7).all()
    start, tab = [0, 4, 6, 9], good.np_table()
    before = Batch("bf16_d64", Hq=2, Hkv=2, page=16, pos=[14, 3, 20], counts=[4, 2, 3], seed=10, max_pos=64)
    for s, (p0, n) in enumerate(zip([14, 3, 20], [4, 2, 3])):
        for i in range(n):
            pg, sl = tab[s][(p0 + i) // 16], (p0 + i) % 16
            if start[s] + i in skipped:
                assert torch.equal(b.k_pages[pg, :, sl], before.k_pages[pg, :, sl])
            else:
                check_rows(b.k_pages[pg, :, sl], k_ref[pg, :, sl], b.ct, top)
                assert np.array_equal(f64(b.v_pages[pg, :, sl]), v_ref[pg, :, sl])


# ---------------------------------------------------------------- attend

def run_attend(kda, b, what="", n_max=None, **kw):
    ref = b.attend_ref(kw.get("scale"), kw.get("window", 0))
    o, lse = b.attend(kda, **kw)
    torch.cuda.synchronize()
    assert kda.last_variant() == "attn_decode" and b.err.item() == 0, what
    n = n_max or max(int(p) + n for p, n in zip(b.pos.tolist(), b.counts))
    check_attend(o, lse, ref, b.dt, b.dk, n, what)
    return o, lse


@pytest.mark.parametrize("form,T", itertools.product(FORMS, [1, 3]))
def test_attend_forms(kda, form, T):
    b = Batch(form, **heads(form), page=16, pos=[0, 5, 126, 300], counts=[T] * 4, seed=11)
    run_attend(kda, b, form)
    run_attend(kda, b, form, packed=False, lse=False)


EDGES = [-1, 0, 14, 15, 16, 30, 31, 32, 62, 63, 64, 126, 127, 128, 129, 254, 255, 256, 1000]


@pytest.mark.parametrize("form,page", [("bf16_d128", 16), ("bf16_d64", 64), ("f32_d128", 32), ("e4m3_d128", 1024),
                                       ("e4m3_d64", 16), ("f32_d64", 128), ("latent", 16), ("latent", 64)])
def test_attend_lengths(kda, form, page):
    """Lengths around every tile and page edge, a row without tokens among them."""
    b = Batch(form, **heads(form, 4, 2), page=page, pos=EDGES, counts=[1] * len(EDGES), seed=12)
    o, lse = run_attend(kda, b, form)
    assert (o[0] == 0).all() and (lse[0] == -float("inf")).all()


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "latent"])
def test_attend_drafts_and_idle_sequences(kda, form):
    b = Batch(form, **heads(form), page=16, pos=[40, -3, 7, 127, 0, 500], counts=[4, 5, 0, 1, 16, 2], seed=13)
    o, lse = run_attend(kda, b, form)
    assert (o[4:6] == 0).all()                           # positions -3 and -2: nothing to see
    o2, _ = b.attend(kda, lse=False)
    assert torch.equal(o, o2), "equal calls give equal bits"


@pytest.mark.parametrize("hq,hkv,T", [(1, 1, 1), (3, 1, 1), (12, 4, 1), (5, 5, 2), (16, 1, 1), (17, 1, 1), (40, 2, 3),
                                      (64, 1, 1), (32, 2, 16), (64, 1, 16), (48, 8, 5)])
@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "e4m3_d64"])
def test_attend_heads(kda, form, hq, hkv, T):
    b = Batch(form, Hq=hq, Hkv=hkv, page=32, pos=[200, 31], counts=[T, T], seed=14)
    run_attend(kda, b, form)


@pytest.mark.parametrize("hq,T", [(1, 1), (8, 2), (16, 1), (17, 3), (32, 4), (64, 2), (128, 1), (33, 16)])
def test_attend_latent_heads(kda, hq, T):
    b = Batch("latent", Hq=hq, Hkv=1, page=64, pos=[200, 31], counts=[T, T], seed=15)
    run_attend(kda, b)


@pytest.mark.parametrize("hq,T", [(64, 2), (24, 5), (16, 4), (33, 1), (32, 16)])
@pytest.mark.parametrize("room", [1600, 6000, 40000, 1 << 18])
def test_attend_latent_row_blocks(kda, hq, T, room):
    """The room of the page table sets how many query rows a workgroup takes: 16 to 128."""
    pos = [1500, 200, 31]
    b = Batch("latent", Hq=hq, Hkv=1, page=64, pos=pos, counts=[T, 0, T], seed=31,
              extra_cols=room // 64 - (1500 + T + 63) // 64)
    o, lse = run_attend(kda, b)
    o2, lse2 = b.attend(kda)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    run_attend(kda, b, "window", window=90, n_max=100)
    ref = b.attend_ref(window=20)
    tab = b.np_table()
    seen = torch.zeros((b.n_pages, 64), dtype=torch.bool)
    for s in (0, 2):
        for p in range(pos[s] + 1 - 20, pos[s] + T):
            seen[tab[s][p // 64], p % 64] = True
    b.k_pages.permute(0, 2, 1, 3)[~seen.to(b.device)] = float("nan")
    o, lse = b.attend(kda, window=20)
    assert b.err.item() == 0
    check_attend(o, lse, ref, b.dt, b.dk, 24 + T, "NaN around")
    if T > 1:                                            # a NaN that only the last new token sees
        b.k_pages[tab[2][(31 + T - 1) // 64], :, (31 + T - 1) % 64] = float("nan")
        o, lse = b.attend(kda, window=20)
        rows = list(range(2 * T - 1))
        check_attend(o[rows], lse[rows], tuple(x[rows] for x in ref), b.dt, b.dk, 24 + T, "NaN in the last token")
        assert o[-1].isnan().all()


@pytest.mark.parametrize("room", [512, 3000, 20000, 1 << 17])
def test_attend_latent_row_blocks_refuse_a_page(kda, room):
    b = Batch("latent", Hq=64, Hkv=1, page=64, pos=[400, 90, 300, 7], counts=[4, 4, 4, 4], seed=32,
              extra_cols=room // 64 - 7)
    ref = b.attend_ref()
    b.table[1, 1] = b.n_pages
    o, lse = b.attend(kda)
    assert b.err.item() == 32
    assert (o[4:8] == 7).all() and (lse[4:8] == 7).all()
    rows = [0, 1, 2, 3] + list(range(8, 16))
    check_attend(o[rows], lse[rows], tuple(x[rows] for x in ref), b.dt, b.dk, 404)


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "e4m3_d64", "latent"])
@pytest.mark.parametrize("window", [1, 2, 17, 128, 1000])
def test_attend_window(kda, form, window):
    b = Batch(form, **heads(form), page=16, pos=[0, 40, 129, 300], counts=[4, 1, 3, 4], seed=16)
    run_attend(kda, b, form, window=window)


@pytest.mark.parametrize("form", ["bf16_d128", "e4m3_d128", "f32_d128", "latent"])
def test_attend_long_contexts_are_split_and_joined(kda, form):
    b = Batch(form, **heads(form, 4, 2), page=64, pos=[6000, 100, 2500, -1], counts=[1, 2, 1, 1], seed=17)
    run_attend(kda, b, form)
    b = Batch(form, **heads(form, 2, 1), page=256, pos=[20000], counts=[1], seed=18)
    run_attend(kda, b, form)


def test_attend_many_sequences(kda):
    rng = np.random.default_rng(1)
    for form in ("bf16_d64", "latent"):
        pos = np.minimum(rng.geometric(0.01, 300), 900)
        b = Batch(form, Hq=2, Hkv=1, page=16, pos=pos, counts=rng.integers(0, 3, 300), seed=19)
        run_attend(kda, b, form)


@pytest.mark.parametrize("B,hq,T", [(60, 32, 4), (150, 16, 2), (66, 64, 3), (200, 1, 1)])
def test_attend_latent_batches_of_uneven_sequences(kda, B, hq, T):
    """Runs of the list of tiles that begin, end and pass over sequences of one tile and of many, idle ones between."""
    rng = np.random.default_rng(B)
    pos = rng.choice([-1, 0, 31, 40, 300, 1300], B, p=[0.05, 0.2, 0.2, 0.3, 0.15, 0.1])
    counts = rng.integers(0, T + 1, B)
    b = Batch("latent", Hq=hq, Hkv=1, page=32, pos=pos, counts=counts, seed=34)
    run_attend(kda, b)
    run_attend(kda, b, "window", window=33, n_max=64)


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "latent"])
def test_attend_scales(kda, form):
    b = Batch(form, **heads(form), page=16, pos=[100, 257], counts=[1, 2], seed=20)
    for scale in (0.0, -0.05, 1.0, 40.0 / b.dk):
        run_attend(kda, b, f"{form} scale {scale}", scale=scale)


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "e4m3_d128", "latent"])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_hidden_tokens_do_not_reach_a_row(kda, form, junk):
    """What lies past the sequence, before the window or at later drafts may hold anything."""
    b = Batch(form, **heads(form), page=16, pos=[37, 130, 5], counts=[3, 4, 1], seed=21)
    ref = b.attend_ref(window=20)
    ks, vs = b.k_pages.clone(), None if b.v_pages is None else b.v_pages.clone()
    seen = torch.zeros((b.n_pages, b.page), dtype=torch.bool)
    tab = b.np_table()
    for s, (p0, n) in enumerate(zip([37, 130, 5], b.counts)):
        for p in range(max(0, p0 + 1 - 20), p0 + n):
            seen[tab[s][p // 16], p % 16] = True
    hidden = ~seen.to(b.device)
    for x in (b.k_pages, b.v_pages):
        if x is not None:
            y = x.float()
            y.permute(0, 2, 1, 3)[hidden] = junk
            x.copy_(y.clamp(-448, 448) if x.dtype == torch.float8_e4m3fn and not np.isnan(junk) else y)
    o, lse = b.attend(kda, window=20)
    assert b.err.item() == 0
    check_attend(o, lse, ref, b.dt, b.dk, 24, "junk around")
    # A later draft's own key and value, seen by itself but not by the rows before it.
    b.k_pages.copy_(ks)
    if vs is not None:
        b.v_pages.copy_(vs)
    for s, p in ((0, 39), (1, 133)):
        for x in (b.k_pages, b.v_pages):
            if x is not None:
                bad = 448.0 if x.dtype == torch.float8_e4m3fn and not np.isnan(junk) else junk
                x[tab[s][p // 16], :, p % 16] = torch.full((), bad, device=b.device).to(x.dtype)
    o2, lse2 = b.attend(kda, window=20)
    rows = [0, 1, 3, 4, 5, 7]
    check_attend(o2[rows], lse2[rows], tuple(x[rows] for x in ref), b.dt, b.dk, 24, "junk in a later draft")
    if np.isnan(junk):
        assert o2[[2, 6]].isnan().all() and lse2[[2, 6]].isnan().all()


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "latent"])
def test_scores_of_minus_infinity(kda, form):
    """Keys of -inf weigh nothing beside others, and make 0 / 0 where a row sees nothing else, as in the formula."""
    b = Batch(form, **heads(form, 4, 2), page=64, pos=[40, 9000, -1], counts=[2, 1, 1], seed=33)
    col, tab = 570 if b.latent else 5, b.np_table()
    b.q[..., col] = 1.0
    one = [(tab[0][0], 7), (tab[1][0], 7)]               # token 7 of both
    keys = [b.k_pages[pg, :, at].clone() for pg, at in one]
    b.k_pages[..., col] = -float("inf")
    o, lse = b.attend(kda)
    assert o[:3].isnan().all() and (o[3] == 0).all() and lse.isneginf().all()
    for (pg, at), key in zip(one, keys):
        b.k_pages[pg, :, at] = key
    o, lse = b.attend(kda)
    assert b.err.item() == 0
    for row, (pg, at) in zip((0, 1, 2), (one[0], one[0], one[1])):
        v = b.k_pages[pg, :, at, :512] if b.latent else b.v_pages[pg, :, at]
        assert torch.equal(o[row], v.repeat_interleave(b.Hq // b.Hkv, 0))
    assert lse[:3].isfinite().all() and (o[3] == 0).all()


@pytest.mark.parametrize("form", ["bf16_d128", "f32_d64", "latent"])
def test_nan_in_a_seen_value_reaches_its_column_only(kda, form):
    b = Batch(form, **heads(form), page=16, pos=[300], counts=[2], seed=22)
    tab = b.np_table()
    ref = b.attend_ref()
    x = b.k_pages if b.latent else b.v_pages
    x[tab[0][100 // 16], :, 100 % 16, 5] = float("nan")
    o, _ = b.attend(kda)
    if b.latent:
        assert o.isnan().all()                           # the key is NaN too
        return
    assert o[..., 5].isnan().all()
    cols = [c for c in range(b.dv) if c != 5]
    check_attend(o[..., cols], None, (ref[0][..., cols], ref[1], ref[2][..., cols], ref[3]), b.dt, b.dk, 302)


@pytest.mark.parametrize("what,bit", [("page", 32), ("page_high", 32), ("table", 32), ("backwards", 128), ("long", 128),
                                      ("past", 128), ("start", 128)])
@pytest.mark.parametrize("form", ["bf16_d64", "latent"])
def test_attend_refuses_on_the_device(kda, what, bit, form):
    """A bad sequence is named and none of its rows written; the others are served."""
    b = Batch(form, **heads(form, 4, 2), page=16, pos=[700, 2000, 30], counts=[2, 2, 3], seed=23)
    ref = b.attend_ref()
    T, bad = 3, range(2, 4)
    if what == "page":
        b.table[1, 60] = -1
    elif what == "page_high":
        b.table[1, 125] = b.n_pages
    elif what == "table":
        b.pos[1] = 16 * b.table.shape[1] - 1
    elif what == "backwards":
        b.tok_start[3], bad = 3, range(4, 7)
    elif what == "long":
        T, bad = 2, range(4, 7)
    elif what == "past":
        b.tok_start[3], bad = 8, range(4, 7)
    else:
        b.tok_start[0], bad = -1, range(0, 2)
    pool = b.pool(kda)
    o, lse = torch.full((7, b.Hq, b.dv), 7.0, dtype=b.dt, device="cuda"), torch.full((7, b.Hq), 7.0, device="cuda")
    ws = kda.attn_workspace(pool, b.table, Hq=b.Hq, T=3)
    kda.attn_decode(pool, b.table, b.pos, b.q, o, ws, b.err, lse=lse, tok_start=b.tok_start, T=T)
    torch.cuda.synchronize()
    assert b.err.item() == bit
    rows = [r for r in range(7) if r not in bad]
    check_attend(o[rows], lse[rows], tuple(x[rows] for x in ref), b.dt, b.dk, 2002, what)
    assert (o[list(bad)] == 7).all() and (lse[list(bad)] == 7).all()


def test_rows_of_no_sequence_are_left_alone(kda):
    b = Batch("bf16_d128", Hq=4, Hkv=2, page=16, pos=[60, 10], counts=[2, 1], seed=24)
    ref = b.attend_ref()
    pool, n = b.pool(kda), 9
    pad = lambda x, v: torch.cat([x, torch.full((n - 3, *x.shape[1:]), v, dtype=x.dtype, device="cuda")])  # noqa: E731
    q, o = pad(b.q, 1.0), torch.full((n, 4, 128), 7.0, dtype=b.dt, device="cuda")
    ws = kda.attn_workspace(pool, b.table, Hq=4, T=2)
    kda.attn_decode(pool, b.table, b.pos, q, o, ws, b.err, tok_start=b.tok_start, T=2)
    check_attend(o[:3], None, ref, b.dt, b.dk, 62)
    assert (o[3:] == 7).all() and b.err.item() == 0
    kp = b.k_pages.clone()
    _, k_ref, _ = b.append_ref()
    q_out = torch.full_like(q, 7.0)
    kda.kv_append(pool, b.table, b.pos, pad(b.k, 1.0), pad(b.v, 1.0), b.err, q=q, q_out=q_out, cos_sin=b.cos_sin,
                  tok_start=b.tok_start, T=2)
    check_rows(b.k_pages, k_ref, b.ct, 10.0)
    assert (q_out[3:] == 7).all() and not torch.equal(kp, b.k_pages) and b.err.item() == 0


def test_attend_strided_queries(kda):
    b = Batch("bf16_d128", Hq=8, Hkv=2, page=16, pos=[300, 90], counts=[3, 3], seed=25)
    o, lse = b.attend(kda)
    wide = torch.zeros((2, 3, 12, 128), dtype=b.dt, device="cuda")
    wide[:, :, :8] = b.dense(b.q)
    o2 = torch.empty((2, 3, 8, 128), dtype=b.dt, device="cuda")
    pool = b.pool(kda)
    kda.attn_decode(pool, b.table, b.pos, wide[:, :, :8], o2, kda.attn_workspace(pool, b.table, Hq=8, T=3), b.err)
    assert torch.equal(o2.view_as(o), o)


@pytest.mark.parametrize("form", ["bf16_d128", "latent"])
def test_attend_far_pages(kda, form):
    """A pool of more than 2^31 values: pages past 4 GiB are reached."""
    page, Hkv, dk = (1024, 8, 128) if form == "bf16_d128" else (1024, 1, 576)
    n_pages = 2200 if form == "bf16_d128" else 3800
    b = Batch(form, Hq=8, Hkv=Hkv, page=page, pos=[1500], counts=[2], seed=26)
    ref = b.attend_ref()
    big = [None if x is None else torch.empty((n_pages, *x.shape[1:]), dtype=x.dtype, device="cuda")
           for x in (b.k_pages, b.v_pages)]
    tab = b.table.clone()
    for i in range(2):
        for x, y in zip(big, (b.k_pages, b.v_pages)):
            if x is not None:
                x[n_pages - 1 - i] = y[int(b.table[0, i])]
        tab[0, i] = n_pages - 1 - i
    pool = kda.PagePool.from_tensors(big[0], big[1], dv=b.dv)
    o, lse = torch.empty((2, 8, b.dv), dtype=b.dt, device="cuda"), torch.empty((2, 8), device="cuda")
    ws = kda.attn_workspace(pool, tab, Hq=8, T=2)
    kda.attn_decode(pool, tab, b.pos, b.q, o, ws, b.err, lse=lse, tok_start=b.tok_start, T=2)
    check_attend(o, lse, ref, b.dt, b.dk, 1502, form)
    kda.kv_append(pool, tab, b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=2)      # not rotated: a copy
    assert torch.equal(big[0][n_pages - 2, :, 1500 - 1024:1502 - 1024].transpose(0, 1), b.k)
    assert b.err.item() == 0


def test_long_position_in_a_long_table(kda):
    """Positions past 2^20 with a window: only the window's pages are read."""
    page, pos = 1024, (1 << 20) + 77
    b = Batch("bf16_d64", Hq=4, Hkv=2, page=page, pos=[1100], counts=[1], seed=27)
    tab = torch.full((1, 1026), -5, dtype=torch.int32, device="cuda")
    tab[0, 1023], tab[0, 1024] = b.table[0, 0], b.table[0, 1]
    b.pos[0] = 1024 + 77                                 # the same places in the small table
    ref = b.attend_ref(window=500)
    b.pos[0] = pos
    b.table = tab
    o, lse = b.attend(kda, window=500)
    assert b.err.item() == 0
    check_attend(o, lse, ref, b.dt, b.dk, 500)


# ---------------------------------------------------------------- streams and graphs

def test_side_stream_and_two_calls_at_once(kda):
    a = Batch("bf16_d128", Hq=8, Hkv=2, page=64, pos=[9000], counts=[1], seed=28)
    c = Batch("latent", Hq=16, Hkv=1, page=64, pos=[5000, 40], counts=[2, 1], seed=29)
    ra, rc = a.attend_ref(), c.attend_ref()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        oa, la = a.attend(kda)
    with torch.cuda.stream(s2):
        oc, lc = c.attend(kda)
    torch.cuda.synchronize()
    check_attend(oa, la, ra, a.dt, a.dk, 9001)
    check_attend(oc, lc, rc, c.dt, c.dk, 5002)


@pytest.mark.parametrize("form", ["bf16_d128", "e4m3_d64", "latent"])
def test_captured_round_replays(kda, form):
    """append + attend captured once; every replay reads the positions of its round, eager work in between."""
    b = Batch(form, **heads(form), page=16, pos=[2000, 33, 0], counts=[2, 0, 1], seed=30)
    rounds = 4
    grow = Batch(form, **heads(form), page=16, pos=[2000 + 8 * rounds, 33 + 8 * rounds, 8 * rounds], counts=[2, 0, 1],
                 seed=30)
    b.k_pages, b.v_pages, b.table, b.n_pages, b.cos_sin = grow.k_pages, grow.v_pages, grow.table, grow.n_pages, grow.cos_sin
    pool = b.pool(kda)
    q_rot, o = torch.empty_like(b.q), torch.empty((3, b.Hq, b.dv), dtype=b.dt, device="cuda")
    lse = torch.empty((3, b.Hq), device="cuda")
    ws = kda.attn_workspace(pool, b.table, Hq=b.Hq, T=2)
    ap = kda.KvAppendPlan(pool, b.table, b.pos, b.k, b.v, b.err, q=b.q, q_out=q_rot, cos_sin=b.cos_sin,
                          rot_start=b.rot_start, tok_start=b.tok_start, T=2)
    at = kda.AttnDecodePlan(pool, b.table, b.pos, q_rot, o, ws, b.err, lse=lse, tok_start=b.tok_start, T=2)
    ap(), at()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ap(), at()
    rng = np.random.default_rng(5)
    for r in range(rounds):
        for t in (b.q, b.k, b.v):
            if t is not None:
                t.copy_(dev_tensor(rng.standard_normal(tuple(t.shape), dtype=np.float32)))
        o.fill_(7), lse.fill_(7), q_rot.fill_(7), ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        got = (o.clone(), lse.clone(), q_rot.clone(), b.k_pages.clone())
        ref = b.attend_ref(q=q_rot)
        check_attend(o, lse, ref, b.dt, b.dk, 2040, f"replay {r}")
        o.fill_(9)
        ap(), at()
        torch.cuda.synchronize()
        for x, y in zip(got, (o, lse, q_rot, b.k_pages)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), f"replay {r} against the eager calls"
        b.pos += torch.tensor([2, 0, 1], device="cuda")
    assert b.err.item() == 0


def test_two_graphs_that_share_a_workspace(kda):
    """Replayed in turn, each gives what it gives alone; a workspace holds nothing between calls."""
    a = Batch("bf16_d128", Hq=8, Hkv=2, page=64, pos=[7000, 300], counts=[2, 4], seed=34)
    c = Batch("bf16_d128", Hq=8, Hkv=2, page=64, pos=[50, 6800], counts=[4, 1], seed=35)
    pa, pc = a.pool(kda), c.pool(kda)
    ws = max((kda.attn_workspace(p, x.table, Hq=8, T=4) for p, x in ((pa, a), (pc, c))), key=torch.Tensor.numel)
    outs, graphs, plans = [], [], []
    for b, p in ((a, pa), (c, pc)):
        o, lse = torch.empty((b.N, 8, 128), dtype=b.dt, device="cuda"), torch.empty((b.N, 8), device="cuda")
        plans.append(kda.AttnDecodePlan(p, b.table, b.pos, b.q, o, ws, b.err, lse=lse, tok_start=b.tok_start, T=4))
        plans[-1]()
        torch.cuda.synchronize()
        outs.append((o, lse))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plans[-1]()
        graphs.append(g)
    refs = [a.attend_ref(), c.attend_ref()]
    for turn in range(3):
        for g, (o, lse), b, ref in zip(graphs, outs, (a, c), refs):
            o.fill_(7), lse.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            check_attend(o, lse, ref, b.dt, b.dk, 7004, f"turn {turn}")
        ws.fill_(turn * 85)


# ---------------------------------------------------------------- beside the recurrent calls

def test_speculative_rounds_of_a_hybrid_stack(kda):
    """Rounds of drafts through an attention layer and a recurrent layer that share `pos`: append, attend and verify
    the drafts, then commit the accepted ones, which moves pos; rejected drafts are written over."""
    B, H, T, rounds = 3, 4, 4, 5
    spec = synth.ConfigSpec("hybrid", 121, (B,), H, 64, 64, "bf16", "softplus", "normal", 0)
    n_tok = rounds * T
    S0 = synth.initial_state(spec, B)
    inp = synth.token_inputs(spec, B, n_tok)
    d = dev_inputs(inp)
    state, pos = dev_tensor(S0), torch.zeros(B, dtype=torch.int64, device="cuda")
    log, err = kda.InputLog(state, T_max=T), torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(3)
    # The attention layer's own projections of every token, and its cache.
    att = Batch("bf16_d64", Hq=8, Hkv=2, page=16, pos=[0] * B, counts=[n_tok] * B, seed=31)
    full = {n: att.dense(getattr(att, n)) for n in ("q", "k", "v")}
    pool = att.pool(kda)
    ws = kda.attn_workspace(pool, att.table, Hq=8, T=T)
    kept = [[] for _ in range(B)]                        # the stream's accepted token of each position
    for r in range(rounds):
        accepted = rng.integers(0, T + 1, B)
        at = [len(x) for x in kept]
        rows = {n: x[:, r * T:(r + 1) * T].contiguous() for n, x in full.items()}
        q_rot, o = torch.empty_like(rows["q"]), torch.empty_like(rows["q"])
        kda.kv_append(pool, att.table, pos, rows["k"], rows["v"], err, q=rows["q"], q_out=q_rot, cos_sin=att.cos_sin)
        kda.attn_decode(pool, att.table, pos, q_rot, o, ws, err)
        dr = {n: x[:, r * T:(r + 1) * T].contiguous() for n, x in d.items()}
        ov = torch.empty((B, T, H, 64), device="cuda")
        kda.verify(state, dr["q"], dr["k"], dr["v"], dr["alpha"], dr["beta"], ov, log)
        kda.commit(state, pos, log, torch.tensor(accepted, dtype=torch.int32, device="cuda"), err)
        # What a plain stack over each sequence's own tokens gives for this round's drafts.
        cs = f64(att.cos_sin)
        from oracle import paged_oracle as po
        for b in range(B):
            toks = kept[b] + list(range(r * T, (r + 1) * T))
            n = len(toks)
            kp, vp = np.zeros((1, 2, 1024, 64)), np.zeros((1, 2, 1024, 64))
            fk, fv, fq = (f64(full[x][b][toks]) for x in ("k", "v", "q"))
            for p in range(n):                           # stored keys are rounded to bf16
                kp[0, :, p] = f64(torch.from_numpy(po.rotate(fk[p], cs[p])).to(torch.bfloat16))
                vp[0, :, p] = fv[p]
            qr = f64(q_rot[b])
            for t in range(T):
                want = po.rotate(fq[at[b] + t], cs[at[b] + t])
                assert np.abs(qr[t] - want).max() <= 2.0 ** -8 * 5
            ref = po.attend(kp, vp, [[0]], [at[b]], [T], qr, 64 ** -0.5)
            # A stored key may differ from the oracle's by its own rounding (a tie that fp32 decides): 2^-7 of it
            # in single values, far below the bf16 terms of the bound.
            check_attend(o[b], None, ref, torch.bfloat16, 64, n, f"round {r} sequence {b}")
            kept[b] += toks[at[b]:at[b] + accepted[b]]
        assert pos.tolist() == [len(x) for x in kept]
    assert err.item() == 0
    for b in range(B):
        sel = {n: x[b:b + 1][:, kept[b]] for n, x in inp.items()}
        S_ref, _ = ko.decode(S0[b:b + 1], sel, spec.scale)
        rel = np.linalg.norm(state[b].cpu().numpy() - S_ref[0]) / np.linalg.norm(S_ref[0])
        say("hybrid sequence", b, "tokens", len(kept[b]), "state error", rel)
        assert rel <= 1e-3


def test_prompt_then_decode(kda):
    """A prompt appended at once, then decoded token by token: the cache of both ways is the same, bit for bit."""
    b = Batch("bf16_d128", Hq=8, Hkv=2, page=32, pos=[0, 0], counts=[70, 70], seed=32)
    pool = b.pool(kda)
    kda.kv_append(pool, b.table, b.pos, b.dense(b.k), b.dense(b.v), b.err, cos_sin=b.cos_sin)
    want = (b.k_pages.clone(), b.v_pages.clone())
    b.k_pages.zero_(), b.v_pages.zero_()
    pos = b.pos.clone()
    for t in range(70):
        k, v = (b.dense(x)[:, t:t + 1].contiguous() for x in (b.k, b.v))
        kda.kv_append(pool, b.table, pos, k, v, b.err, cos_sin=b.cos_sin)
        pos += 1
    used = torch.zeros((b.n_pages, 32), dtype=torch.bool, device="cuda")
    for s in range(2):
        for p in range(70):
            used[b.table[s, p // 32].long(), p % 32] = True
    for x, y in zip(want, (b.k_pages, b.v_pages)):
        assert torch.equal(x.transpose(1, 2)[used], y.transpose(1, 2)[used])
    assert b.err.item() == 0


def test_other_device_or_host_tensors_are_refused(kda):
    b = Batch("bf16_d64", Hq=2, Hkv=1, page=16, pos=[3], counts=[1], seed=33)
    pool = b.pool(kda)
    o, ws = torch.empty((1, 2, 64), dtype=b.dt, device="cuda"), kda.attn_workspace(pool, b.table, Hq=2)
    for bad in (b.q.cpu(), b.q.half()):
        with pytest.raises((ValueError, TypeError)):
            kda.attn_decode(pool, b.table, b.pos, bad, o, ws, b.err, tok_start=b.tok_start, T=1)
    with pytest.raises(ValueError):
        kda.kv_append(pool, b.table.cpu(), b.pos, b.k, b.v, b.err, tok_start=b.tok_start, T=1)
    with pytest.raises(kda.KdaError):
        kda.attn_decode(pool, b.table, b.pos, b.q, o, ws[:0], b.err, tok_start=b.tok_start, T=1)
