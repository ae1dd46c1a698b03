"""The calls on the paged cache with pages past 2^32 bytes of a pool: bit for bit what a small pool gives, on the GPU."""

from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, PAGE, BLOCK = 3, 16, 8, 128, 64, 32
SMALL = 40


@pytest.fixture(scope="module")
def kda():
    import recurrent_state_amd as k
    k.lib()
    return k


def one_round(kda, pool, pages, form, keep):
    """Append with axes, attend, weigh, evict; what all of these left, in the pages that `pages` names."""
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(3)
    table, dst = pages[:30].view(B, 10).contiguous(), pages[30:39].view(B, 3).contiguous()
    pos = torch.tensor([500, 33, 601], device=dev)
    T = 3
    q, k, v = (torch.randn((B, T, h, D), device=dev, generator=g).bfloat16() for h in (HQ, HKV, HKV))
    ang = torch.randn((700, D), device=dev, generator=g)
    axis_pos = torch.randint(0, 700, (2, B, T), device=dev, generator=g)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kda.kv_append(pool, table, pos, k, v, err, q=q, q_out=q, cos_sin=ang, axis_pos=axis_pos,
                  axis_of=kda.rotation_axes([20, 44]))
    o, lse = torch.empty_like(q), torch.empty((B, T, HQ), device=dev)
    ws = kda.attn_workspace(pool, table, Hq=HQ, T=T)
    kda.attn_decode(pool, table, pos, q, o, ws, err, lse=lse)
    weights = torch.rand((B, HKV, 640), device=dev, generator=g)
    kda.attn_weights(pool, table, pos, q, lse, weights, err)
    wide = torch.randn((B, 40, HQ, D), device=dev, generator=g).bfloat16()
    many = torch.full((B, 40, HQ), 6.0, device=dev)
    more = torch.zeros_like(weights)
    if form == "blocks":  # and the rows of a prompt's end, over places below the table's end
        kda.attn_weights(pool, table, pos - 33, wide, many, more, err)
    length, new_w = pos + T, torch.empty_like(weights)
    kept = torch.empty((B, HKV, keep), dtype=torch.int32, device=dev)
    kda.kv_evict(pool, table, length, weights, dst, length, new_w, kept, err, recent=10)
    torch.cuda.synchronize()
    assert err.item() == 0
    at = pages[:39].long()
    got = [q, o, lse, weights, more, new_w, kept, length, pool.k[at].view(torch.uint8), pool.v[at].view(torch.uint8)]
    return got + ([pool.k_scale[at], pool.v_scale[at]] if form == "blocks" else [])


@pytest.mark.parametrize("form", ["bf16", "blocks"])
def test_pages_past_32_bit_offsets(kda, form):
    dev = torch.device("cuda")
    dtype = torch.float8_e4m3fn if form == "blocks" else torch.bfloat16
    es = 1 if form == "blocks" else 2
    n_large = (1 << 32) // (HKV * PAGE * D * es) + 50
    g = torch.Generator(dev).manual_seed(1)
    k0, v0 = (torch.randn((SMALL, HKV, PAGE, D), device=dev, generator=g).to(dtype) for _ in range(2))
    s0 = [2.0 ** torch.randint(-8, -3, (SMALL, HKV, PAGE // BLOCK), device=dev, generator=g) for _ in range(2)]
    high = torch.randperm(n_large - SMALL, device=dev, generator=g)[:SMALL].to(torch.int32)
    high[:SMALL:2] = torch.arange(n_large - SMALL // 2, n_large, dtype=torch.int32, device=dev)  # every other past 2^32 bytes
    assert high.unique().numel() == SMALL
    got = []
    for ids, n in ((torch.arange(SMALL, dtype=torch.int32, device=dev), SMALL), (high, n_large)):
        at = ids.long()
        k, v = (torch.empty((n, HKV, PAGE, D), dtype=dtype, device=dev) for _ in range(2))
        k.view(torch.uint8)[at], v.view(torch.uint8)[at] = k0.view(torch.uint8), v0.view(torch.uint8)
        kw = {}
        if form == "blocks":
            scales = [torch.ones((n, HKV, PAGE // BLOCK), device=dev) for _ in range(2)]
            for x, y in zip(scales, s0):
                x[at] = y
            kw = dict(k_scale=scales[0], v_scale=scales[1], scale_block=BLOCK)
        got.append(one_round(kda, kda.PagePool.from_tensors(k, v, **kw), ids, form, keep=150))
        del k, v, kw
    for x, y in zip(*got):
        assert torch.equal(x, y)
