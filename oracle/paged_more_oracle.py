"""fp64 oracle of the further paged cache calls: rotation by positions on several axes, e4m3 pages with scales by blocks
of tokens, sums of attention weights, and eviction by them.

Plain NumPy over one token, block or head at a time, on the layouts of paged_oracle.py; shares no code with the GPU path.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import paged_oracle as po


def axis_row(cos_sin, at, axis_of):
    """The cosines and sines ([dim]: halves) that a token's pairs turn by: pair n at position at[axis_of[n]]."""
    half = len(axis_of)
    c = [cos_sin[at[a]][n] for n, a in enumerate(axis_of)]
    s = [cos_sin[at[a]][half + n] for n, a in enumerate(axis_of)]
    return np.array(c + s, dtype=np.float64)


def rotated(rows, at, cos_sin, axis_of=None, start=0, pairs=False):
    """Token rows [N][heads][d], row r turned by its position(s) at[r] (a number, or one for each axis)."""
    out = [po.rotate(x, cos_sin[p] if axis_of is None else axis_row(cos_sin, p, axis_of), start, pairs)
           for x, p in zip(rows, at)]
    return np.array(out).reshape(np.shape(rows))


def block_scale(m):
    """The least power of two, 2^-64 or more, with m <= 448 of it."""
    if m == 0:
        return 2.0 ** -64
    part, e = math.frexp(m)  # m = part 2^e, part in [0.5, 1); 448 = 0.875 2^9
    return 2.0 ** max(-64, e - 9 + (part > 0.875))


def append_blocks(pages, scales, table, pos, counts, rows, block):
    """Writes token rows (already rotated) into pages [n_pages][Hkv][page][d] of one side, fp64 arrays in place, and their
    blocks' scales.  What is written is the value that an 8-bit page rounds: clip(x / scale, +-448), and for a block's
    earlier tokens old * (old scale / new scale).  Returns the largest finite magnitude of each touched block and head."""
    page_size, top, row = pages.shape[2], {}, 0
    for b, n in enumerate(counts):
        at = 0
        while at < n:
            p = int(pos[b]) + at
            past = min(n, at + block - p % block)
            page, slot = table[b][p // page_size], p % page_size
            k, held = slot // block, slot % block
            for h in range(pages.shape[1]):
                x = np.asarray(rows[row + at:row + past, h], np.float64)
                fin = np.abs(x[np.isfinite(x)])
                m = top[page, h, k] = float(fin.max()) if fin.size else 0.0
                s = block_scale(m)
                if held:
                    old = scales[page, h, k]
                    s = max(s, 2.0 ** math.ceil(math.log2(old)))
                    pages[page, h, k * block:slot] *= old / s
                scales[page, h, k] = s
                pages[page, h, slot:slot + past - at] = np.clip(x / s, -448, 448)
            at = past
        row += n
    return top


def unscaled(pages, scales, block):
    """The values that pages with scales by blocks stand for."""
    return np.asarray(pages, np.float64) * np.repeat(np.asarray(scales, np.float64), block, axis=2)[..., None]


def weigh(k_pages, table, pos, counts, q, lse, weights, scale, window=0):
    """(weights, terms, spread): the sums after the call, what the call added to each, and the largest size of the terms
    that made one of its scores; all [B][Hkv][places]."""
    w, added, spread = weights.astype(np.float64), np.zeros(weights.shape), np.zeros(weights.shape)
    Hkv, page_size = k_pages.shape[1:3]
    G = q.shape[1] // Hkv
    row = 0
    for b, n in enumerate(counts):
        for j in range(max(0, int(pos[b])), int(pos[b]) + n):
            w[b, :, j] = 0
        for i in range(n):
            p = int(pos[b]) + i
            j = np.arange(max(0, p + 1 - window) if window else 0, p + 1)
            at = np.asarray(table[b])[j // page_size], j % page_size
            for h in range(q.shape[1]):
                k = k_pages[at[0], h // G, at[1]].astype(np.float64)
                e = np.exp(scale * (k @ q[row, h].astype(np.float64)) - float(lse[row, h]))
                added[b, h // G, j] += e
                spread[b, h // G, j] = np.maximum(spread[b, h // G, j],
                                                  abs(scale) * (np.abs(k) @ np.abs(q[row, h].astype(np.float64))))
            row += 1
    return w + added, added, spread


def keep_places(weights, length, keep, recent):
    """The places that one kv head of a sequence of `length` tokens keeps, ascending."""
    if length <= keep:
        return list(range(length))
    cut = length - recent
    rank = sorted(range(cut), key=lambda j: (math.isnan(weights[j]), -weights[j] if weights[j] == weights[j] else 0, j))
    return sorted(rank[:keep - recent]) + list(range(cut, length))
