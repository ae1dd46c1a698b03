"""What an eviction's plan refuses beside wrong shapes and types (meta tensors)."""

from __future__ import annotations

import pytest
import torch

from tests.test_pages_host import _FakePool, _meta, k  # noqa: F401


def plan(k, keep, recent, pages=3):  # noqa: F811
    pool, table, pos, err = _FakePool(k), _meta(2, 4, dtype=torch.int32), _meta(2, dtype=torch.int64), _meta(1, dtype=torch.int32)
    w, new_w = (_meta(2, 2, 256, dtype=torch.float32) for _ in range(2))
    return k.KvEvictPlan(pool, table, pos, w, _meta(2, pages, dtype=torch.int32), pos, new_w,
                         _meta(2, 2, keep, dtype=torch.int32), err, recent=recent)


@pytest.mark.parametrize("keep,recent,pages", [(0, 0, 3), (193, 0, 3), (65, 10, 1), (1, 2, 3), (100, 101, 3), (100, -1, 3)])
def test_budgets_that_no_call_takes(k, keep, recent, pages):  # noqa: F811
    with pytest.raises(ValueError):
        plan(k, keep, recent, pages)


@pytest.mark.parametrize("keep,recent,pages", [(1, 0, 1), (1, 1, 1), (64, 64, 1), (192, 5, 3)])
def test_budgets_at_the_limits(k, keep, recent, pages):  # noqa: F811
    assert plan(k, keep, recent, pages) is not None
