"""Refusals of the further paged cache calls on the host: the C ABI (fake pointers that never reach a device) and the
binding (meta tensors)."""

from __future__ import annotations

import ctypes

import pytest
import torch

from tests.test_pages_host import (ALIGN, BAD_SHAPES, BF16, DTYPE, E4M3, F32, GOOD, MIS, NULL, OK, P, SHAPE, _FakePool,  # noqa: F401
                                   _meta, k, pages, shp)

ref = ctypes.byref


def rotation(k, cs=0x10000, mp=64, start=0, dim=128, pairs=0):  # noqa: F811
    return k._lib._Rotation(cs, mp, start, dim, pairs)


def axes(k, pos=0x10000, stride=0, n=3, of=bytes([0, 1, 2, 0] * 16)):  # noqa: F811
    return k._lib._Axes(pos, stride, n, of)


def scales(k, ks=0x10000, vs=0x10000, block=64):  # noqa: F811
    return k._lib._BlockScales(ks, vs, block)


def opt(x):
    return None if x is None else ref(x)


def app_axes(k, s=None, pg=None, ts=None, N=8, q=None, qo=None, rot="good", ax="good", **kw):  # noqa: F811
    s, pg = s or shp(k), pg or pages(k)
    rot, ax = rotation(k) if rot == "good" else rot, axes(k) if ax == "good" else ax
    a = dict(table=GOOD, cols=4, pos=GOOD, kp=GOOD, kst=0, v=GOOD, vst=0, err=GOOD) | kw
    return k.lib().kda_kv_append_axes(ref(s), ref(pg), a["table"], a["cols"], ts, N, a["pos"], a["kp"], a["kst"], a["v"],
                                      a["vst"], q, 0, qo, 0, opt(rot), opt(ax), a["err"], None)


def app_blocks(k, s=None, pg=None, sc="good", ts=None, N=8, q=None, qo=None, rot=None, ax=None, **kw):  # noqa: F811
    s, pg, sc = s or shp(k, ct=E4M3), pg or pages(k), scales(k) if sc == "good" else sc
    a = dict(table=GOOD, cols=4, pos=GOOD, kp=GOOD, kst=0, v=GOOD, vst=0, err=GOOD) | kw
    return k.lib().kda_kv_append_blocks(ref(s), ref(pg), opt(sc), a["table"], a["cols"], ts, N, a["pos"], a["kp"], a["kst"],
                                        a["v"], a["vst"], q, 0, qo, 0, opt(rot), opt(ax), a["err"], None)


def att_blocks(k, s=None, pg=None, sc="good", ts=None, N=8, **kw):  # noqa: F811
    s, pg, sc = s or shp(k, ct=E4M3), pg or pages(k), scales(k) if sc == "good" else sc
    a = dict(table=GOOD, cols=4, pos=GOOD, q=GOOD, qst=0, scale=0.1, window=0, o=GOOD, lse=GOOD, ws=GOOD, nws=1 << 40,
             err=GOOD) | kw
    return k.lib().kda_attn_decode_blocks(ref(s), ref(pg), opt(sc), a["table"], a["cols"], ts, N, a["pos"], a["q"], a["qst"],
                                          a["scale"], a["window"], a["o"], a["lse"], a["ws"], a["nws"], a["err"], None)


def weigh(k, s=None, pg=None, sc=None, ts=None, N=8, **kw):  # noqa: F811
    s, pg = s or shp(k), pg or pages(k)
    a = dict(table=GOOD, cols=4, pos=GOOD, q=GOOD, qst=0, scale=0.1, window=0, lse=GOOD, w=GOOD, stride=256, err=GOOD) | kw
    return k.lib().kda_attn_weights(ref(s), ref(pg), opt(sc), a["table"], a["cols"], ts, N, a["pos"], a["q"], a["qst"],
                                    a["scale"], a["window"], a["lse"], a["w"], a["stride"], a["err"], None)


def evict(k, s=None, pg=None, sc=None, **kw):  # noqa: F811
    s, pg = s or shp(k), pg or pages(k)
    a = dict(table=GOOD, cols=4, len=GOOD, w=GOOD, stride=256, keep=100, recent=10, dst=GOOD, dcols=2, new_len=GOOD,
             new_w=GOOD, kept=GOOD, err=GOOD) | kw
    return k.lib().kda_kv_evict(ref(s), ref(pg), opt(sc), a["table"], a["cols"], a["len"], a["w"], a["stride"], a["keep"],
                                a["recent"], a["dst"], a["dcols"], a["new_len"], a["new_w"], a["kept"], a["err"], None)


ALL = [app_axes, app_blocks, att_blocks, weigh, evict]


@pytest.mark.parametrize("f", ALL)
@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_shapes(k, f, kw):  # noqa: F811
    s = shp(k, **(kw | (dict(ct=E4M3) if "blocks" in f.__name__ else {})))
    more = {} if f is evict else dict(N=max(0, s.B * s.T))
    assert f(k, s, **more) == SHAPE


@pytest.mark.parametrize("f", ALL)
def test_pointers(k, f):  # noqa: F811
    for name in ("table", "err", "len" if f is evict else "pos"):
        assert f(k, **{name: None}) == NULL
        assert f(k, **{name: P(0x10001)}) == ALIGN
    for name in {app_axes: ("kp", "v"), app_blocks: ("kp", "v"), att_blocks: ("q", "o", "ws"), weigh: ("q", "lse", "w"),
                 evict: ("w", "dst", "new_len", "new_w", "kept")}[f]:
        assert f(k, **{name: None}) == NULL, name
        assert f(k, **{name: P(0x10001)}) == ALIGN, name
    assert f(k, pg=pages(k, kp=None)) == NULL and f(k, pg=pages(k, vp=0x10008)) == ALIGN
    assert f(k, cols=0) == SHAPE and f(k, cols=1 << 26) == SHAPE and f(k, pg=pages(k, n=0)) == SHAPE


def test_axes(k):  # noqa: F811
    assert app_axes(k, rot=None) == NULL and app_axes(k, ax=None) == NULL
    assert app_axes(k, ax=axes(k, pos=None)) == NULL and app_axes(k, ax=axes(k, of=None)) == NULL
    assert app_axes(k, ax=axes(k, pos=0x10004)) == ALIGN
    for bad in (axes(k, n=0), axes(k, n=5), axes(k, stride=7), axes(k, stride=-8), axes(k, stride=1 << 41),
                axes(k, of=bytes([0, 1, 3, 0] * 16)), axes(k, of=bytes([255] * 64)), axes(k, n=1)):
        assert app_axes(k, ax=bad) == SHAPE
    assert app_axes(k, rot=rotation(k, mp=0)) == SHAPE and app_axes(k, rot=rotation(k, dim=24)) == SHAPE
    assert app_axes(k, q=GOOD) == NULL and app_axes(k, rot=rotation(k, cs=None)) == NULL
    e4 = shp(k, ct=E4M3)
    assert app_axes(k, e4) == NULL                          # scales by heads, as kda_kv_append
    assert app_axes(k, shp(k, B=0), N=0, table=None, pos=None, err=None, kp=None, v=None) == OK


@pytest.mark.parametrize("f", [app_blocks, att_blocks, weigh, evict])
def test_block_scales(k, f):  # noqa: F811
    e4 = shp(k, ct=E4M3)
    for block in (0, 8, 24, 128, -64, 1 << 30):
        assert f(k, e4, sc=scales(k, block=block)) == SHAPE
    assert f(k, e4, pages(k, size=1024), sc=scales(k, block=512), **({"keep": 9} if f is evict else {}),
             **({"stride": 1 << 12} if f in (weigh, evict) else {})) == SHAPE
    assert f(k, e4, sc=scales(k, ks=None)) == NULL and f(k, e4, sc=scales(k, vs=None)) == NULL
    assert f(k, e4, sc=scales(k, ks=0x10002)) == ALIGN
    assert f(k, shp(k), sc=scales(k)) == DTYPE and f(k, shp(k, dt=F32, ct=F32), sc=scales(k)) == DTYPE
    if f in (app_blocks, att_blocks):
        assert f(k, sc=None) == NULL
    else:
        assert f(k, e4, sc=None) == NULL                    # scales by heads are not there either


def test_blocks_are_for_the_grouped_form(k):  # noqa: F811
    lat = shp(k, Hkv=1, dk=576, dv=512, ct=E4M3)
    for f in (app_blocks, att_blocks, weigh, evict):
        assert f(k, lat, pages(k, vp=None), sc=scales(k)) == DTYPE


def test_weights_arguments(k):  # noqa: F811
    assert weigh(k, stride=255) == SHAPE and weigh(k, stride=-1) == SHAPE and weigh(k, stride=1 << 33) == SHAPE
    assert weigh(k, shp(k, T=129), N=258) == SHAPE and weigh(k, shp(k, T=128), N=256, q=None) == NULL
    assert weigh(k, window=-1) == SHAPE and weigh(k, scale=float("nan")) == SHAPE and weigh(k, qst=1000) == SHAPE
    assert weigh(k, shp(k, Hkv=1, dk=576, dv=512), pages(k, vp=None)) == SHAPE
    assert weigh(k, shp(k, B=64), N=256, cols=1 << 24, stride=1 << 30) == SHAPE
    assert weigh(k, ts=GOOD, N=0, q=None, lse=None, w=None) == OK


def test_evict_arguments(k):  # noqa: F811
    for bad in (dict(keep=0), dict(keep=129), dict(recent=-1), dict(recent=101), dict(dcols=0), dict(dcols=1 << 26),
                dict(stride=255), dict(stride=1 << 33)):
        assert evict(k, **bad) == SHAPE, bad
    assert evict(k, shp(k, B=1 << 18, T=1 << 10, Hq=8, Hkv=8)) == SHAPE
    assert evict(k, shp(k, Hkv=1, dk=576, dv=512), pages(k, vp=None), w=None) == NULL   # latent pools are taken
    # new_weights in weights (B * Hkv * stride floats), and a table that names its own pages.
    s, at = shp(k, B=2, T=1, Hq=8, Hkv=4), lambda i: type(GOOD)(GOOD.value + i)  # noqa: E731
    for i in (0, 4 * 8 * 512 - 4, 4 - 4 * 8 * 512):
        assert evict(k, s, new_w=at(i), stride=512, dst=at(4096)) == SHAPE
    assert evict(k, s, new_w=at(4 * 8 * 512), stride=512) == SHAPE
    assert evict(k, shp(k, Hkv=1, dk=576, dv=512)) == SHAPE
    none = dict(table=None, len=None, w=None, dst=None, new_len=None, new_w=None, kept=None, err=None)
    assert evict(k, shp(k, B=0), pages(k, None, None), **none) == OK
    assert k.lib().kda_kv_evict(None, None, None, GOOD, 4, GOOD, GOOD, 256, 100, 10, GOOD, 2, GOOD, GOOD, GOOD, GOOD,
                                None) == NULL


# ---------------------------------------------------------------- the binding

def test_rotation_axes(k):  # noqa: F811
    assert k.rotation_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert k.rotation_axes([2, 1, 3], interleaved=True) == [0, 1, 2, 0, 2, 2]
    for bad in ([], [1] * 5, [2, -1]):
        with pytest.raises(ValueError):
            k.rotation_axes(bad)


def test_binding_of_axes(k):  # noqa: F811
    pool, table, pos, err = _FakePool(k), _meta(2, 4, dtype=torch.int32), _meta(2, dtype=torch.int64), _meta(1, dtype=torch.int32)
    kk, v, cs = _meta(2, 3, 2, 128), _meta(2, 3, 2, 128), _meta(64, 128, dtype=torch.float32)
    of = k.rotation_axes([30, 34])
    ap = lambda **kw: k.KvAppendPlan(pool, table, pos, kk, v, err, **kw)  # noqa: E731
    at = lambda *shape, dtype=torch.int64: _meta(*shape, dtype=dtype)  # noqa: E731
    ap(cos_sin=cs, axis_pos=at(2, 2, 3), axis_of=of)
    ap(cos_sin=cs, axis_pos=at(1, 2, 3))
    for kw, exc in [(dict(axis_pos=at(2, 2, 3), axis_of=of), ValueError),                       # no table
                    (dict(cos_sin=cs, axis_of=of), ValueError), (dict(cos_sin=cs, axis_pos=at(2, 2, 3)), ValueError),
                    (dict(cos_sin=cs, axis_pos=at(2, 6), axis_of=of), ValueError),
                    (dict(cos_sin=cs, axis_pos=at(2, 2, 3, dtype=torch.int32), axis_of=of), TypeError),
                    (dict(cos_sin=cs, axis_pos=at(5, 2, 3), axis_of=of), ValueError),
                    (dict(cos_sin=cs, axis_pos=at(2, 2, 3), axis_of=of[:-1]), ValueError),
                    (dict(cos_sin=cs, axis_pos=at(2, 2, 3), axis_of=[2] * 64), ValueError),
                    (dict(cos_sin=cs, axis_pos=[1, 2], axis_of=of), TypeError)]:
        with pytest.raises(exc):
            ap(**kw)


def test_binding_of_weights_and_evictions(k):  # noqa: F811
    pool, table, pos, err = _FakePool(k), _meta(2, 4, dtype=torch.int32), _meta(2, dtype=torch.int64), _meta(1, dtype=torch.int32)
    q, lse, w = _meta(2, 3, 8, 128), _meta(2, 3, 8, dtype=torch.float32), _meta(2, 2, 256, dtype=torch.float32)
    k.AttnWeightsPlan(pool, table, pos, q, lse, w, err)
    for args, exc in [((q, lse[:, :, :4], w), ValueError), ((q, lse.bfloat16(), w), TypeError), ((q, lse, w[:, :, :255]), ValueError),
                      ((q, lse, w[:, :1]), ValueError), ((q, lse, w.double()), TypeError),
                      ((q, lse, _meta(2, 256, 2, dtype=torch.float32).transpose(1, 2)), ValueError), ((q, lse, None), TypeError)]:
        with pytest.raises(exc):
            k.AttnWeightsPlan(pool, table, pos, *args, err)
    dst, kept = _meta(2, 3, dtype=torch.int32), _meta(2, 2, 100, dtype=torch.int32)
    k.KvEvictPlan(pool, table, pos, w, dst, pos, w, kept, err, recent=3)
    for args, exc in [((w, dst[:1], pos, w, kept), ValueError), ((w, dst.long(), pos, w, kept), TypeError),
                      ((w, dst, pos.int(), w, kept), TypeError), ((w, dst, pos, w[:, :, :200], kept), ValueError),
                      ((w, dst, pos, w, kept[:, 0]), ValueError), ((w, dst, pos, w, kept.long()), TypeError)]:
        with pytest.raises(exc):
            k.KvEvictPlan(pool, table, pos, *args, err)


def test_binding_of_block_pools(k):  # noqa: F811
    for kw in (dict(dtype=torch.bfloat16), dict(scale_block=8), dict(scale_block=48), dict(scale_block=128)):
        with pytest.raises(ValueError):
            k.PagePool(4, 64, 2, 128, 128, "cpu", **(dict(dtype=torch.float8_e4m3fn, scale_block=16) | kw))
