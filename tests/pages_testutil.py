"""Seeded paged caches for the tests of the paged attention calls, and the error bounds that they use."""

from __future__ import annotations

import numpy as np
import torch

from oracle import paged_oracle as po

FORMS = {  # name: (dk, dv, in dtype, cache dtype)
    "bf16_d128": (128, 128, torch.bfloat16, torch.bfloat16),
    "bf16_d64": (64, 64, torch.bfloat16, torch.bfloat16),
    "f32_d128": (128, 128, torch.float32, torch.float32),
    "f32_d64": (64, 64, torch.float32, torch.float32),
    "e4m3_d128": (128, 128, torch.bfloat16, torch.float8_e4m3fn),
    "e4m3_d64": (64, 64, torch.bfloat16, torch.float8_e4m3fn),
    "latent": (576, 512, torch.bfloat16, torch.bfloat16),
}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
TINY_STEP = {torch.bfloat16: 0.0, torch.float32: 0.0, torch.float8_e4m3fn: 2.0 ** -10}  # half of the subnormal step


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


class Batch:
    """Pages, a table and token rows of one call; `pos` tokens are cached, counts[b] are new."""

    def __init__(self, form, *, Hq, Hkv, page, pos, counts, seed=0, device="cuda", spare=2, extra_cols=0, fill=None,
                 max_pos=None, rot_dim=None):
        self.form, self.Hq, self.Hkv, self.page, self.counts = form, Hq, Hkv, page, list(counts)
        self.dk, self.dv, self.dt, self.ct = FORMS[form]
        self.latent = form == "latent"
        rng = np.random.default_rng(seed)
        dev = self.device = torch.device(device)
        B, N = len(pos), sum(counts)
        self.B, self.N, self.T = B, N, max(max(counts, default=1), 1)
        need = [max(0, -(-(p + n) // page)) for p, n in zip(pos, counts)]
        n_pages = sum(need) + spare
        ids = rng.permutation(n_pages)
        table, at = np.full((B, max(max(need), 1) + extra_cols), -1, np.int32), 0
        for b, k in enumerate(need):
            table[b, :k], at = ids[at:at + k], at + k
        self.n_pages = n_pages

        def dev_t(x, dtype):
            return torch.from_numpy(np.ascontiguousarray(x)).to(dev).to(dtype)

        def pages(width):
            x = dev_t(rng.standard_normal((n_pages, Hkv, page, width), dtype=np.float32), torch.float32)
            if fill is not None:
                x.fill_(fill)
            return (x * 8).to(self.ct) if self.ct == torch.float8_e4m3fn else x.to(self.ct)

        self.k_pages = pages(self.dk)
        self.v_pages = None if self.latent else pages(self.dv)
        self.k_scale = self.v_scale = None
        if self.ct == torch.float8_e4m3fn:
            self.k_scale = dev_t(0.1 * (1 + rng.random(Hkv)), torch.float32)
            self.v_scale = dev_t(0.1 * (1 + rng.random(Hkv)), torch.float32)
        self.table = dev_t(table, torch.int32)
        self.pos = dev_t(np.asarray(pos, np.int64), torch.int64)
        self.tok_start = dev_t(np.concatenate([[0], np.cumsum(counts)]), torch.int32)
        self.q = dev_t(rng.standard_normal((N, Hq, self.dk), dtype=np.float32), self.dt)
        self.k = dev_t(rng.standard_normal((N, Hkv, self.dk), dtype=np.float32), self.dt)
        self.v = None if self.latent else dev_t(rng.standard_normal((N, Hkv, self.dv), dtype=np.float32), self.dt)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.rot_start = self.dv if self.latent else 0
        dim = rot_dim or (64 if self.latent else self.dk)
        max_pos = max_pos or max([p + n for p, n in zip(pos, counts)] + [1])
        ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
        self.cos_sin = dev_t(np.concatenate([np.cos(ang), np.sin(ang)], 1), torch.float32)

    def pool(self, kda):
        return kda.PagePool.from_tensors(self.k_pages, self.v_pages, dv=self.dv, k_scale=self.k_scale,
                                         v_scale=self.v_scale)

    def dense(self, x):
        return x.view(self.B, self.T, *x.shape[1:])

    def np_table(self):
        return self.table.cpu().numpy()

    # -------------------------------------------------------------- expected results

    def append_ref(self, pairs=False, rotated=True, with_q=True):
        kp, vp = f64(self.k_pages), f64(self.v_pages)
        q = po.append(kp, vp, self.np_table(), self.pos.cpu().numpy(), self.counts, f64(self.k), f64(self.v),
                      f64(self.q) if with_q else None, f64(self.cos_sin) if rotated else None, self.rot_start, pairs,
                      f64(self.k_scale), f64(self.v_scale))
        return q, kp, vp

    def attend_ref(self, scale=None, window=0, q=None):
        return po.attend(f64(self.k_pages), f64(self.v_pages), self.np_table(), self.pos.cpu().numpy(), self.counts,
                         f64(self.q if q is None else q), self.dk ** -0.5 if scale is None else scale, window,
                         f64(self.k_scale), f64(self.v_scale), self.dv)

    def attend(self, kda, *, scale=None, window=0, packed=True, lse=True, ws=None, q=None, o=None, pool=None):
        pool = pool or self.pool(kda)
        q = self.q if q is None else q
        o = torch.full((self.N, self.Hq, self.dv), 7.0, dtype=self.dt, device=self.device) if o is None else o
        out_l = torch.full((self.N, self.Hq), 7.0, device=self.device) if lse else None
        ws = kda.attn_workspace(pool, self.table, Hq=self.Hq, T=self.T) if ws is None else ws
        if packed:
            kda.attn_decode(pool, self.table, self.pos, q, o, ws, self.err, lse=out_l, scale=scale, window=window,
                            tok_start=self.tok_start, T=self.T)
        else:
            kda.attn_decode(pool, self.table, self.pos, self.dense(q), self.dense(o), ws, self.err,
                            lse=self.dense(out_l) if lse else None, scale=scale, window=window)
        return o, out_l


def check_rows(got, want, dtype, terms=None, what=""):
    """got within a rounding of want: half a step of the stored type, plus four fp32 roundings of the terms
    (two products, their sum, and the division by an 8-bit scale) that made it."""
    g, w = f64(got), np.asarray(want)
    t = np.abs(w) if terms is None else np.maximum(terms, np.abs(w))
    # A stored value was rounded from one that four fp32 roundings had moved.
    tol = HALF_STEP[dtype] * np.abs(w) + TINY_STEP[dtype] + 4 * 2.0 ** -24 * t * (1 + HALF_STEP[dtype])
    bad = ~(np.abs(g - w) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(g - w)[bad].max()}"


def attend_bounds(ref, dtype, dk, n_max):
    """Bounds of |o - o_ref| and |lse - lse_ref| from the roundings made.

    A score is a sum of dk products (exact in fp32 for bf16 inputs, else one rounding each) and dk additions, times
    scale, log2 e and an 8-bit scale: at most ds = (2 dk + 4) 2^-24 of its terms' sum, a change of e^s by the factor
    e^(+-2 ds) against the others.  The exponential adds 2^-22 and the sums n 2^-24.  bf16 outputs round the
    probabilities to bf16 once (half a step, 2^-8, each: it averages out, but this bounds it) and the result once.
    """
    o, lse, weight, spread = ref
    ds = (2 * dk + 4) * 2.0 ** -24 * spread
    rel = 2 * ds + 2.0 ** -21 + (n_max + 64) * 2.0 ** -24
    half = HALF_STEP[dtype]
    prob = half if dtype == torch.bfloat16 else 0.0
    o_tol = half * np.abs(o) + (1 + half) * (prob + rel)[..., None] * weight
    lse_tol = rel + 4 * 2.0 ** -24 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + ds
    return o_tol, lse_tol


def check_attend(o, lse, ref, dtype, dk, n_max, what=""):
    o_tol, lse_tol = attend_bounds(ref, dtype, dk, max(n_max, 1))
    d = np.abs(f64(o) - ref[0])
    assert (d <= o_tol).all(), f"{what}: o off by {d.max():.3e}, {(~(d <= o_tol)).sum()} of {d.size} over the bound"
    if lse is not None:
        g, w = f64(lse), ref[1]
        empty = np.isneginf(w)
        assert (np.isneginf(g) == empty).all(), f"{what}: rows without tokens"
        dl = np.where(empty, 0.0, np.abs(np.where(empty, 0, g) - np.where(empty, 0, w)))
        assert (dl <= lse_tol).all(), f"{what}: lse off by {dl.max():.3e}"
