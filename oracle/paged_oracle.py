"""fp64 oracle of the paged attention cache: appending rotated keys and values, and attending to them.

Plain NumPy over one sequence, head and token at a time; shares no code with the GPU path.  Pages are
[n_pages][Hkv][page_size][width], a table row lists a sequence's pages in order, token i of a sequence's new tokens
sits at position pos + i.  A latent cache passes v_pages = None: a key row's first dv values are its value.
"""

from __future__ import annotations

import numpy as np


def rotate(x, cos_sin_row, start=0, pairs=False):
    """x [..., dk] with the values from `start` on rotated by one position's cosines and sines ([dim]: halves)."""
    x = np.array(x, dtype=np.float64)
    half = len(cos_sin_row) // 2
    c, s = np.asarray(cos_sin_row[:half], np.float64), np.asarray(cos_sin_row[half:], np.float64)
    n = np.arange(half)
    i, j = (start + 2 * n, start + 2 * n + 1) if pairs else (start + n, start + half + n)
    xi, xj = x[..., i], x[..., j]
    x[..., i], x[..., j] = xi * c - xj * s, xj * c + xi * s
    return x


def append(k_pages, v_pages, table, pos, counts, k, v, q=None, cos_sin=None, start=0, pairs=False, k_scale=None,
           v_scale=None):
    """Writes the new tokens' rows into k_pages and v_pages (fp64 arrays, in place) and returns the rotated queries.

    counts[b] tokens of sequence b are the next rows of k, v and q.  With scales, what is written is
    clip(x / scale, +-448): the value an 8-bit page rounds.
    """
    page_size = k_pages.shape[2]
    q_out = None if q is None else np.array(q, dtype=np.float64)
    row = 0
    for b, n in enumerate(counts):
        for i in range(n):
            p = int(pos[b]) + i
            page, slot = table[b][p // page_size], p % page_size
            kr = np.asarray(k[row], np.float64) if cos_sin is None else rotate(k[row], cos_sin[p], start, pairs)
            k_pages[page, :, slot] = kr if k_scale is None else np.clip(kr / k_scale[:, None], -448, 448)
            if v is not None:
                vr = np.asarray(v[row], np.float64)
                v_pages[page, :, slot] = vr if v_scale is None else np.clip(vr / v_scale[:, None], -448, 448)
            if q is not None:
                q_out[row] = rotate(q[row], cos_sin[p], start, pairs)
            row += 1
    return q_out


def attend(k_pages, v_pages, table, pos, counts, q, scale, window=0, k_scale=None, v_scale=None, dv=None):
    """(o [N][Hq][dv], lse [N][Hq], weight [N][Hq][dv], spread [N][Hq]) of the new tokens' queries.

    weight is sum_j p_j |v_j| (what a relative error of the probabilities can move o by) and spread
    max_j scale sum_d |q_d k_jd| (the size of the terms that make a score).
    """
    N, Hq, _ = q.shape
    Hkv, page_size = k_pages.shape[1:3]
    dv = v_pages.shape[-1] if v_pages is not None else dv
    o, weight = np.zeros((N, Hq, dv)), np.zeros((N, Hq, dv))
    lse, spread = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    row = 0
    for b, n in enumerate(counts):
        for i in range(n):
            p = int(pos[b]) + i
            lo = max(0, p + 1 - window) if window else 0
            if p >= 0:
                j = np.arange(lo, p + 1)
                at = (np.asarray(table[b])[j // page_size], j % page_size)
                for h in range(Hq):
                    hk = h // (Hq // Hkv)
                    kr = k_pages[at[0], hk, at[1]].astype(np.float64)
                    vr = kr[:, :dv] if v_pages is None else v_pages[at[0], hk, at[1]].astype(np.float64)
                    if k_scale is not None:
                        kr, vr = kr * float(k_scale[hk]), vr * float(v_scale[hk])
                    qr = q[row, h].astype(np.float64)
                    s = scale * (kr @ qr)
                    m = s.max()
                    e = np.exp(s - m)
                    o[row, h] = (e @ vr) / e.sum()
                    weight[row, h] = (e @ np.abs(vr)) / e.sum()
                    lse[row, h] = m + np.log(e.sum())
                    spread[row, h] = abs(scale) * (np.abs(kr) @ np.abs(qr)).max()
            row += 1
    return o, lse, weight, spread
