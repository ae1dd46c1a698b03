"""The paged attention calls on the host: argument checks of the C ABI (fake pointers that never reach a device) and
of the binding.  Runs with or without a GPU; nothing is launched."""

from __future__ import annotations

import ctypes
import os

import pytest
import torch

OK, NULL, SHAPE, DTYPE, ALIGN = 0, 1, 2, 3, 4
P = ctypes.c_void_p
GOOD, MIS = P(0x10000), P(0x10004)
BF16, F32, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def k():
    import recurrent_state_amd as kda
    if not os.path.exists(kda.LIB_PATH):
        from recurrent_state_amd import build
        build.build()
    return kda


def shp(k, B=2, T=4, Hq=8, Hkv=2, dk=128, dv=128, dt=BF16, ct=BF16):
    return k.KvShape(B, T, Hq, Hkv, dk, dv, dt, ct)


def pages(k, kp=0x10000, vp=0x10000, ks=None, vs=None, n=4, size=64):
    return k._lib._Pages(kp, vp, ks, vs, n, size)


def app(k, s=None, pg=None, table=GOOD, cols=4, ts=None, N=8, pos=GOOD, kr=GOOD, kst=0, v=GOOD, vst=0, q=None, qst=0,
        qo=None, qost=0, rot=None, err=GOOD):
    s, pg = s or shp(k), pg or pages(k)
    return k.lib().kda_kv_append(ctypes.byref(s), ctypes.byref(pg), table, cols, ts, N, pos, kr, kst, v, vst, q, qst, qo,
                                 qost, None if rot is None else ctypes.byref(rot), err, None)


def att(k, s=None, pg=None, table=GOOD, cols=4, ts=None, N=8, pos=GOOD, q=GOOD, qst=0, scale=0.1, window=0, o=GOOD,
        lse=GOOD, ws=GOOD, nws=1 << 40, err=GOOD):
    s, pg = s or shp(k), pg or pages(k)
    return k.lib().kda_attn_decode(ctypes.byref(s), ctypes.byref(pg), table, cols, ts, N, pos, q, qst, scale, window, o,
                                   lse, ws, nws, err, None)


BAD_SHAPES = [dict(B=-1), dict(T=0), dict(Hkv=0), dict(Hq=0), dict(Hq=7), dict(dk=96, dv=96), dict(dk=128, dv=64),
              dict(dk=64, dv=128), dict(dk=256, dv=256), dict(dk=576, dv=512), dict(Hq=8192)]


@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_shapes(k, kw):
    s = shp(k, **kw)
    N = max(0, s.B * s.T)
    assert app(k, s, N=N) == SHAPE and att(k, s, N=N) == SHAPE
    assert k.lib().kda_attn_workspace_bytes(ctypes.byref(s), ctypes.byref(pages(k)), 4) == 0


@pytest.mark.parametrize("dt,ct", [(E4M3, E4M3), (BF16, F32), (F32, BF16), (F32, E4M3), (5, 5), (BF16, 7)])
def test_types(k, dt, ct):
    assert app(k, shp(k, dt=dt, ct=ct)) == DTYPE and att(k, shp(k, dt=dt, ct=ct)) == DTYPE
    assert att(k, shp(k, Hkv=1, dk=576, dv=512, dt=F32, ct=F32)) == DTYPE
    assert att(k, shp(k, Hkv=1, dk=576, dv=512, ct=E4M3)) == DTYPE


@pytest.mark.parametrize("size", [0, 8, 24, 100, 2048, -64])
def test_page_sizes(k, size):
    assert app(k, pg=pages(k, size=size)) == SHAPE and att(k, pg=pages(k, size=size)) == SHAPE


def test_tables_and_tokens(k):
    for f in (app, att):
        assert f(k, cols=0) == SHAPE and f(k, cols=1 << 26) == SHAPE          # 2^32 positions
        assert f(k, pg=pages(k, n=-1)) == SHAPE
        assert f(k, N=7) == SHAPE and f(k, N=-1) == SHAPE                     # without tok_start: B * T
        assert f(k, table=None) == NULL and f(k, pos=None) == NULL and f(k, err=None) == NULL
        assert f(k, pg=pages(k, kp=None)) == NULL and f(k, pg=pages(k, vp=None)) == NULL
        assert f(k, table=P(0x10002)) == ALIGN and f(k, pos=MIS) == ALIGN and f(k, err=P(0x10001)) == ALIGN
        assert f(k, ts=P(0x10002)) == ALIGN and f(k, pg=pages(k, kp=0x10004)) == ALIGN
        assert f(k, pg=pages(k, vp=0x10008)) == ALIGN
        e4 = shp(k, ct=E4M3)
        assert f(k, e4, pages(k)) == NULL                                     # 8-bit pages need scales
        assert f(k, e4, pages(k, ks=0x10000, vs=0x10002)) == ALIGN
        lat = shp(k, Hkv=1, dk=576, dv=512)
        assert f(k, lat, pages(k)) == SHAPE                                   # a latent pool has no value pages
    assert k.lib().kda_kv_append(None, None, GOOD, 4, None, 8, GOOD, GOOD, 0, GOOD, 0, None, 0, None, 0, None, GOOD,
                                 None) == NULL


def test_launches_fit_the_grid(k):
    s = shp(k, B=1, T=1 << 26)                            # 96 units of 16 values to a token
    most = ((1 << 32) - 256) // 96
    for N in (most + 1, 1 << 26):
        assert app(k, s, ts=GOOD, N=N) == SHAPE
    assert app(k, s, ts=GOOD, N=most, kr=None) == NULL    # passes that check, and is stopped at the next one
    many = shp(k, B=(1 << 20) + 1, T=1)
    assert att(k, many, ts=GOOD, N=8, cols=1) == SHAPE
    assert k.lib().kda_attn_workspace_bytes(ctypes.byref(many), ctypes.byref(pages(k)), 1) == 0
    assert att(k, shp(k, B=1 << 20, T=1), ts=GOOD, N=8, cols=1, q=None) == NULL


def test_append_arguments(k):
    rot = lambda cs=0x10000, mp=64, start=0, dim=128, pairs=0: k._lib._Rotation(cs, mp, start, dim, pairs)  # noqa: E731
    assert app(k, kr=None) == NULL and app(k, v=None) == NULL
    assert app(k, q=GOOD, rot=rot()) == NULL and app(k, qo=GOOD, rot=rot()) == NULL   # both or neither
    assert app(k, q=GOOD, qo=GOOD) == NULL                                    # queries need a rotation
    assert app(k, rot=rot(cs=None)) == NULL and app(k, rot=rot(cs=0x10008)) == ALIGN
    for bad in (rot(mp=0), rot(dim=0), rot(dim=24), rot(dim=144), rot(start=8), rot(start=-16), rot(start=64),
                rot(start=112, dim=32)):
        assert app(k, rot=bad) == SHAPE
    assert app(k, kr=MIS) == ALIGN and app(k, v=MIS) == ALIGN
    assert app(k, kst=255) == SHAPE and app(k, kst=260) == ALIGN and app(k, vst=-256) == SHAPE
    assert app(k, q=GOOD, qo=GOOD, rot=rot(), qst=1023) == SHAPE and app(k, q=GOOD, qo=MIS, rot=rot()) == ALIGN
    lat = shp(k, Hkv=1, dk=576, dv=512)
    assert app(k, lat, pages(k, vp=None)) == SHAPE                            # values with a latent pool


def test_attend_arguments(k):
    assert att(k, q=None) == NULL and att(k, o=None) == NULL
    assert att(k, q=MIS) == ALIGN and att(k, o=MIS) == ALIGN and att(k, lse=P(0x10002)) == ALIGN
    assert att(k, shp(k, T=17), N=34) == SHAPE and att(k, window=-1) == SHAPE
    assert att(k, scale=float("inf")) == SHAPE and att(k, scale=float("nan")) == SHAPE
    assert att(k, qst=1000) == SHAPE and att(k, qst=1028) == ALIGN
    need = k.lib().kda_attn_workspace_bytes(ctypes.byref(shp(k)), ctypes.byref(pages(k)), 4)
    assert need > 0
    assert att(k, ws=None) == NULL and att(k, nws=255) == SHAPE and att(k, ws=P(0x10080)) == ALIGN


@pytest.mark.parametrize("kw", [dict(Hq=8, Hkv=2), dict(Hq=64, Hkv=1), dict(Hq=32, Hkv=32), dict(Hq=24, Hkv=8, dt=F32, ct=F32),
                                dict(Hq=32, Hkv=1, dk=576, dv=512), dict(Hq=128, Hkv=1, dk=576, dv=512)])
def test_a_workspace_serves_calls_with_fewer_tokens(k, kw):
    sizes = [k.lib().kda_attn_workspace_bytes(ctypes.byref(shp(k, B=5, T=t, **kw)), ctypes.byref(pages(k)), 300)
             for t in range(1, 17)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_positions_are_bounded(k):
    assert k.lib().kda_attn_workspace_bytes(ctypes.byref(shp(k, B=64)), ctypes.byref(pages(k)), 1 << 24) == 0
    assert att(k, shp(k, B=64, T=4), N=256, cols=1 << 24) == SHAPE            # 2^36 tokens


def test_nothing_to_do(k):
    before = k.lib().kda_last_variant()
    empty = shp(k, B=0)
    none = dict(table=None, pos=None, err=None, N=0, pg=pages(k, None, None))
    assert app(k, empty, kr=None, v=None, **none) == OK and att(k, empty, q=None, o=None, ws=None, nws=0, **none) == OK
    assert app(k, ts=GOOD, N=0) == OK and att(k, ts=GOOD, N=0) == OK          # packed rows, none this call
    assert k.lib().kda_last_variant() == before


# ---------------------------------------------------------------- the binding (meta tensors: no device)

def test_binding_refuses_host_memory(k):
    with pytest.raises(ValueError, match="device memory"):
        k.PagePool(4, 64, 2, 128, 128, "cpu")


class _FakePool:
    """Stands in for a pool where only its sizes matter."""

    def __init__(self, k, latent=False, dtype=torch.bfloat16, dk=128, dv=128, Hkv=2):
        self.k = torch.empty((4, Hkv, 64, dk), dtype=dtype, device="meta")
        self.v = None if latent else torch.empty((4, Hkv, 64, dv), dtype=dtype, device="meta")
        self.Hkv, self.dk, self.dv, self.page_size, self.latent = Hkv, dk, dv, 64, latent
        self.device, self.c = self.k.device, k._lib._Pages(0, 0, 0, 0, 4, 64)


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_checks(k):
    pool = _FakePool(k)
    table, pos, err = _meta(2, 4, dtype=torch.int32), _meta(2, dtype=torch.int64), _meta(1, dtype=torch.int32)
    kk, v, q = _meta(2, 3, 2, 128), _meta(2, 3, 2, 128), _meta(2, 3, 8, 128)
    cs, ts = _meta(64, 128, dtype=torch.float32), _meta(3, dtype=torch.int32)
    ap = lambda *a, **kw: k.KvAppendPlan(pool, *a, **kw)  # noqa: E731
    ap(table, pos, kk, v, err, q=q, q_out=_meta(2, 3, 8, 128), cos_sin=cs)    # the good call builds
    for args, kw, exc in [
        ((table, pos, kk, None, err), {}, ValueError), ((table, pos, kk, _meta(2, 3, 2, 64), err), {}, ValueError),
        ((table, pos, kk, v.float(), err), {}, TypeError), ((table.long(), pos, kk, v, err), {}, TypeError),
        ((table, pos.int(), kk, v, err), {}, TypeError), ((table, pos, kk, v, err), dict(q=q), ValueError),
        ((table, pos, kk, v, err), dict(q=q, q_out=q), ValueError),           # no rotation
        ((table, pos, kk, v, err), dict(tok_start=ts, T=3), ValueError),      # packed rows are [N][H][d]
        ((table, pos, kk[0], v[0], err), dict(tok_start=ts), ValueError),     # T missing
        ((table, pos, kk, v, err), dict(T=4), ValueError),
        ((table, pos, _meta(2, 3, 128, 2).transpose(2, 3), v, err), {}, ValueError),
        ((table, pos, _meta(3, 2, 2, 128).transpose(0, 1), v, err), {}, ValueError),   # token-major
        ((table, pos, kk.half(), v.half(), err), {}, TypeError), ((table[0], pos, kk, v, err), {}, ValueError),
        ((table, pos, kk, v, _meta(2, dtype=torch.int32)), {}, ValueError),
    ]:
        with pytest.raises(exc):
            ap(*args, **kw)
    qkv = _meta(2, 3, 12, 128)                                                 # slices of one projection
    plan = ap(table, pos, qkv[:, :, 8:10], qkv[:, :, 10:], err, q=qkv[:, :, :8], q_out=qkv[:, :, :8], cos_sin=cs)
    assert plan._args[8] == plan._args[10] == plan._args[12] == plan._args[14] == 12 * 128
    ws = _meta(256, dtype=torch.uint8)
    at = lambda qq, o, **kw: k.AttnDecodePlan(pool, table, pos, qq, o, ws, err, **kw)  # noqa: E731
    at(q, _meta(2, 3, 8, 128), lse=_meta(2, 3, 8, dtype=torch.float32))
    for qq, o, kw, exc in [(q, _meta(2, 3, 8, 64), {}, ValueError), (q, _meta(2, 3, 8, 128).float(), {}, TypeError),
                           (q, _meta(2, 3, 8, 128), dict(lse=_meta(2, 3, 8)), TypeError),
                           (q, _meta(2, 3, 8, 128), dict(lse=_meta(2, 8, 3, dtype=torch.float32)), ValueError),
                           (q[0], _meta(3, 8, 128), dict(tok_start=ts), ValueError)]:
        with pytest.raises(exc):
            at(qq, o, **kw)
    with pytest.raises(ValueError):
        k.attn_workspace(pool, table, Hq=8, T=17)
