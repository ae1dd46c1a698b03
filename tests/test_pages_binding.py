"""The binding of the paged attention calls, without a device (meta tensors)."""

from __future__ import annotations

import warnings

import pytest
import torch

from tests.test_pages_host import _FakePool, _meta, k  # noqa: F401  (k: a fixture)


def attend(k, pool, **kw):  # noqa: F811
    table, pos, err = _meta(2, 4, dtype=torch.int32), _meta(2, dtype=torch.int64), _meta(1, dtype=torch.int32)
    q, o, ws = _meta(2, 3, 8, pool.dk), _meta(2, 3, 8, pool.dv), _meta(256, dtype=torch.uint8)
    return k.AttnDecodePlan(pool, table, pos, q, o, ws, err, **kw)


def test_a_latent_cache_asks_for_its_scale(k):  # noqa: F811
    """Its key width is not the width that the model trained with, so the usual default is named when taken."""
    latent = _FakePool(k, latent=True, dk=576, dv=512, Hkv=1)
    with pytest.warns(UserWarning, match="scale"):
        plan = attend(k, latent)
    assert plan._args[9] == 576 ** -0.5
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert attend(k, latent, scale=192 ** -0.5)._args[9] == 192 ** -0.5
        assert attend(k, latent, scale=576 ** -0.5)._args[9] == 576 ** -0.5
        assert attend(k, _FakePool(k))._args[9] == 128 ** -0.5      # grouped heads: the keys' own width
