"""Limits of the paged attention calls on the host, each call's own (fake pointers that never reach a device)."""

from __future__ import annotations

import pytest

from tests.test_pages_host import GOOD, NULL, SHAPE, app, att, k, shp  # noqa: F401  (k: a fixture)


@pytest.mark.parametrize("kw", [dict(Hq=4096, Hkv=4096, B=1 << 16, T=1), dict(Hq=64, Hkv=8, B=1 << 20, T=16),
                                dict(Hq=4096, Hkv=1, dk=64, dv=64, B=1 << 18, T=4)])
def test_attention_has_no_thread_to_each_unit(k, kw):  # noqa: F811
    """2^32 threads are an append's limit; attention takes as many rows as its own limits allow."""
    s = shp(k, **kw)
    N = s.B * s.T
    assert app(k, s, N=N, cols=1) == SHAPE
    assert att(k, s, N=N, cols=1, q=None) == NULL         # past every check of sizes
    assert att(k, s, N=N + 1, cols=1) == SHAPE
