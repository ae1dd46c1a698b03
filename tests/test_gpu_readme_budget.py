"""The serving loop with a budget of tokens that the introduction for users prints, run as it is printed: the sums of
weights follow their tokens through a cut."""

from __future__ import annotations

import os
import textwrap

import numpy as np
import pytest
import torch

from oracle import paged_more_oracle as mo
from tests.conftest import ROOT
from tests.pages_testutil import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def printed_loop():
    """The indented lines after the paragraph on budgets."""
    with open(os.path.join(ROOT, "README.md")) as f:
        lines = f.read().split("A budget of tokens for each head", 1)[1].split("\n")
    first = next(i for i, x in enumerate(lines) if x.startswith("    "))
    last = next((i for i in range(first, len(lines)) if not lines[i].startswith("    ")), len(lines))
    return compile(textwrap.dedent("\n".join(lines[first:last])), "README.md", "exec")


def test_sums_go_on_after_a_cut(kda):
    dev, B, T, Hq, Hkv, d, page, keep, wide = "cuda", 2, 16, 4, 2, 64, 16, 160, 20
    g = torch.Generator(dev).manual_seed(1)
    ang = torch.arange(400)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    tables = torch.arange(2 * B * wide, dtype=torch.int32, device=dev).view(2, B, wide)
    x = dict(kda=kda, torch=torch, T=T, pool=kda.PagePool(2 * B * wide, page, Hkv, d, d, dev), table=tables[0],
             new_table=tables[1], cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().to(dev),
             length=torch.tensor([64, 0], device=dev),       # the first one's earlier keys are zeros, with sums of zero
             err=torch.zeros(1, dtype=torch.int32, device=dev), o=torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device=dev),
             lse=torch.empty((B, T, Hq), device=dev), weights=torch.zeros((B, Hkv, wide * page), device=dev),
             new_weights=torch.full((B, Hkv, wide * page), 7.0, device=dev),
             kept=torch.empty((B, Hkv, keep), dtype=torch.int32, device=dev))
    x["ws"] = kda.attn_workspace(x["pool"], x["table"], Hq=Hq, T=T)
    loop = printed_loop()
    sums, tol, at = np.zeros((B, Hkv, wide * page)), np.zeros((B, Hkv, wide * page)), x["length"].clone()
    for step in range(13):
        x["q"], x["k"], x["v"] = (torch.randn((B, T, h, d), device=dev, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        x["positions"], x["due"] = at[:, None] + torch.arange(T, device=dev), step in (8, 11)
        table, pos = x["table"].cpu().numpy(), x["length"].cpu().numpy()
        exec(loop, x)
        torch.cuda.synchronize()
        at += T
        lse = f64(x["lse"]).reshape(B * T, Hq)
        sums, added, spread = mo.weigh(f64(x["pool"].k), table, pos, [T] * B, f64(x["q"]).reshape(B * T, Hq, d), lse, sums, d ** -0.5)
        # The roundings of tests/test_gpu_weights.py's check, of every step so far.
        err = (2 * d + 4) * 2.0 ** -24 * spread + 2.0 ** -22 * (np.abs(lse).max() + spread)
        tol += (2 * err + 2.0 ** -22 + (T * Hq // Hkv + 8) * 2.0 ** -24) * added + 2.0 ** -23 * np.abs(sums)
        if x["due"]:
            n, kept = pos + T, x["kept"].cpu().numpy()
            for b in range(B):
                assert x["length"][b].item() == min(n[b], keep)
                if n[b] > keep:
                    for h in range(Hkv):
                        s, t = sums[b, h, kept[b, h]], tol[b, h, kept[b, h]]
                        sums[b, h], tol[b, h] = 0, 0
                        sums[b, h, :keep], tol[b, h, :keep] = s, t
        assert (np.abs(f64(x["weights"]) - sums) <= tol).all(), step
    # The first sequence was cut twice, the other once: at the first one it was short.
    assert x["err"].item() == 0 and (x["table"] == torch.stack([tables[0, 0], tables[1, 1]])).all()
