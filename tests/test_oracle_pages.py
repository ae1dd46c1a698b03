"""Pins of the paged-attention oracle: closed forms and invariants (CPU)."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import paged_oracle as po


def _cos_sin(n, dim, seed=0):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_keeps_norms_and_depends_on_distance_only(pairs):
    rng = np.random.default_rng(0)
    cs = _cos_sin(64, 32)
    q, k = rng.standard_normal((2, 48))
    rq = [po.rotate(q, cs[p], 16, pairs) for p in range(64)]
    rk = [po.rotate(k, cs[p], 16, pairs) for p in range(64)]
    assert np.array_equal(rq[0], q)                                   # angle 0
    assert np.allclose([np.linalg.norm(x) for x in rq], np.linalg.norm(q), rtol=1e-14)
    assert all(np.array_equal(x[:16], q[:16]) for x in rq)            # outside the rotated span
    assert np.allclose([rq[p + 7] @ rk[p] for p in range(50)], rq[7] @ rk[0], atol=1e-12)


def test_rotation_by_a_quarter_turn_swaps_each_pair():
    x = np.arange(8.0)
    quarter = np.concatenate([np.zeros(4), np.ones(4)])               # cos 0, sin 1
    assert np.array_equal(po.rotate(x, quarter), [-4, -5, -6, -7, 0, 1, 2, 3])
    assert np.array_equal(po.rotate(x, quarter, pairs=True), [-1, 0, -3, 2, -5, 4, -7, 6])


def _cache(rng, B, pos, counts, page=4, Hkv=2, d=8):
    need = [-(-(p + n) // page) for p, n in zip(pos, counts)]
    table, at = np.full((B, max(need)), -1), 0
    ids = rng.permutation(sum(need))
    for b, k in enumerate(need):
        table[b, :k], at = ids[at:at + k], at + k
    return table, np.zeros((sum(need), Hkv, page, d)), np.zeros((sum(need), Hkv, page, d))


def test_append_one_by_one_equals_append_at_once():
    rng = np.random.default_rng(1)
    cs = _cos_sin(32, 8)
    table, k1, v1 = _cache(rng, 2, [3, 0], [5, 9])
    k2, v2 = k1.copy(), v1.copy()
    k, v, q = rng.standard_normal((3, 14, 2, 8))
    q1 = po.append(k1, v1, table, [3, 0], [5, 9], k, v, q, cs)
    q2 = np.zeros_like(q1)
    for b, (p0, n, r0) in enumerate([(3, 5, 0), (0, 9, 5)]):
        for i in range(n):
            r = r0 + i
            counts = [int(b == 0), int(b == 1)]
            q2[r] = po.append(k2, v2, table, [p0 + i if b == 0 else 0, p0 + i if b == 1 else 0], counts, k[r:r + 1],
                              v[r:r + 1], q[r:r + 1], cs)[0]
    assert np.array_equal(k1, k2) and np.array_equal(v1, v2) and np.array_equal(q1, q2)


def test_equal_scores_average_the_values_and_a_window_of_one_copies_the_own_value():
    rng = np.random.default_rng(2)
    table, k, v = _cache(rng, 1, [9], [2])
    v[:] = rng.standard_normal(v.shape)
    flat = v.swapaxes(1, 2)[table[0]].reshape(-1, 2, 8)               # [token][head][d]
    q = rng.standard_normal((2, 4, 8))
    o, lse, _, _ = po.attend(k, v, table, [9], [2], q, 0.5)           # zero keys: all scores 0
    for h in range(4):
        assert np.allclose(o[0, h], flat[:10, h // 2].mean(0)) and np.allclose(o[1, h], flat[:11, h // 2].mean(0))
    assert np.allclose(lse, np.log([[10] * 4, [11] * 4]))
    o1, lse1, _, _ = po.attend(k, v, table, [9], [2], q, 0.5, window=1)
    assert np.allclose(o1[1, 3], flat[10, 1]) and np.allclose(lse1, 0)


def test_rows_without_tokens_are_zero_and_latent_values_are_the_keys_head():
    rng = np.random.default_rng(3)
    table, k, _ = _cache(rng, 1, [0], [3], Hkv=1)
    k[:] = rng.standard_normal(k.shape)
    q = rng.standard_normal((3, 2, 8))
    o, lse, _, _ = po.attend(k, None, table, [-1], [3], q, 1.0, dv=5)
    assert not o[0].any() and np.isneginf(lse[0]).all()
    assert np.allclose(o[1], k[table[0][0], 0, 0, :5])                # one visible token: its value
    o2, _, _, _ = po.attend(k, k[..., :5], table, [-1], [3], q, 1.0)
    assert np.array_equal(o, o2)
