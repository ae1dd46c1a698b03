"""Pins of the oracle of the further paged cache calls: closed forms and invariants."""

from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import paged_more_oracle as mo
from oracle import paged_oracle as po


def test_one_axis_or_equal_positions_are_the_plain_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 32))
    ang = np.arange(40)[:, None] * 100.0 ** (-np.arange(0, 32, 2) / 32)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    at = rng.integers(0, 40, 5)
    plain = mo.rotated(x, at, cs)
    of = rng.integers(0, 3, 16)
    assert np.array_equal(mo.rotated(x, [[p] * 3 for p in at], cs, of), plain)
    for r, p in enumerate(at):
        assert np.array_equal(plain[r], po.rotate(x[r], cs[p]))


def test_axes_turn_their_own_pairs_only():
    x = np.ones((1, 1, 8))
    ang = np.arange(10)[:, None] * np.ones(4)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = mo.rotated(x, [[0, 3]], cs, [0, 1, 0, 1])[0, 0]
    c, s = math.cos(3), math.sin(3)
    assert np.allclose(y, [1, c - s, 1, c - s, 1, c + s, 1, c + s])


@pytest.mark.parametrize("m,e", [(448, 0), (np.nextafter(448, 500), 1), (449, 1), (896, 1), (7, -6), (1e-30, -64),
                                 (0, -64), (3.4e38, 120), (448 * 2.0 ** -64, -64), (449 * 2.0 ** -64, -63)])
def test_block_scale(m, e):
    assert mo.block_scale(m) == 2.0 ** e


def test_append_blocks_fits_and_raises():
    pages, scales = np.zeros((2, 1, 32, 4)), np.ones((2, 1, 2))
    pages[1, 0, 16:18] = 100.0  # two tokens of value 100 at places 16, 17 of the sequence
    rows = np.full((20, 1, 4), 900.0)
    top = mo.append_blocks(pages, scales, [[1, 0]], [18], [20], rows, 16)
    assert top == {(1, 0, 1): 900.0, (0, 0, 0): 900.0}
    assert scales[1, 0].tolist() == [1, 4] and scales[0, 0].tolist() == [4, 1]  # 900 > 448 * 2
    assert (pages[1, 0, 16:18] == 25).all() and (pages[1, 0, 18:] == 225).all() and (pages[0, 0, :6] == 225).all()
    assert (mo.unscaled(pages, scales, 16)[1, 0, 16:18] == 100).all()
    assert (pages[0, 0, 6:] == 0).all()


def test_a_scale_does_not_fall_while_a_block_holds_earlier_tokens():
    pages, scales = np.zeros((1, 1, 16, 2)), np.full((1, 1, 1), 3.0)
    mo.append_blocks(pages, scales, [[0]], [5], [1], np.full((1, 1, 2), 1.0), 16)
    assert scales[0, 0, 0] == 4.0  # not a power of two: rounded up
    mo.append_blocks(pages, scales, [[0]], [0], [1], np.full((1, 1, 2), 1.0), 16)
    assert scales[0, 0, 0] == mo.block_scale(1.0)


def test_weights_of_a_row_sum_to_one():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((4, 2, 16, 8))
    q = rng.standard_normal((3, 4, 8))
    table, pos, counts = [[2, 0], [1, 3]], [20, 4], [2, 1]
    _, lse, _, _ = po.attend(k, k, table, pos, counts, q, 0.3)
    w0 = rng.random((2, 2, 32))
    w, added, _ = mo.weigh(k, table, pos, counts, q, lse, w0, 0.3)
    assert np.allclose(added.sum(-1), [[4, 4], [2, 2]])  # rows times query heads of a kv head
    assert np.array_equal(w[0, :, 22:], w0[0, :, 22:]) and np.array_equal(w[1, :, 5:], w0[1, :, 5:])
    assert np.allclose(w[0, :, :20], w0[0, :, :20] + added[0, :, :20]) and np.allclose(w[0, :, 20:22], added[0, :, 20:22])
    _, lse, _, _ = po.attend(k, k, table, pos, counts, q, 0.3, 7)
    w, added, _ = mo.weigh(k, table, pos, counts, q, lse, w0, 0.3, 7)
    assert (added[0, :, :14] == 0).all() and np.allclose(added.sum(-1), [[4, 4], [2, 2]])


def test_keep_places():
    w = [5.0, 1.0, math.nan, 5.0, 0.0, -1.0, math.inf, 2.0]
    assert mo.keep_places(w, 8, 8, 2) == list(range(8))
    assert mo.keep_places(w, 8, 3, 1) == [0, 6, 7]          # of the two fives the earlier
    assert mo.keep_places(w, 8, 3, 3) == [5, 6, 7]
    assert mo.keep_places(w, 8, 7, 0) == [0, 1, 3, 4, 5, 6, 7]  # NaN goes first
    assert mo.keep_places([-0.0, 0.0, 0.0], 3, 2, 0) == [0, 1]
