"""More operators on the paged attention cache: what is timed, and their plain forms.

Image and video tokens have a position on each of several axes, a cache in 8 bits is half the
size of one in 16, and a cache of bounded size keeps the tokens that are attended to:

  axes    new keys and values go to their pages, and keys and queries are rotated by several
          positions of their token, one to each group of a head's value pairs
  append  the same into e4m3 pages with one power-of-two scale for each `block` tokens of a kv
          head: a new block gets the smallest scale that holds its values, one that holds
          earlier tokens is raised to it, and those tokens are stored anew
  attend  attention of new tokens over such pages
  weigh   the attention weight that each cached token gets from the new tokens' queries, summed
          over them and over the query heads of its kv head, is added to its sum so far; a new
          token's own sum begins at zero
  evict   of a sequence longer than `keep`, each kv head's last `recent` tokens and the others
          of the greatest sums, `keep` in all, move in order to the places 0, 1, ... of other
          pages, and their sums with them

Layouts: queries, keys and values are packed token rows [N][heads][width], sequence b owning rows
tok_start[b] .. tok_start[b + 1] - 1 at places pos[b], pos[b] + 1, ...; the cache holds
[pages][kv heads][page size][width]; table[b][i] is the page with places i * page size and on.
Scales of blocks are [pages][kv heads][page size / block], sums of weights [B][kv heads][places].

With `own` false, run() computes the plain forms from elementary torch operations in 32 bits;
with `own` true it makes the library's calls.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TABLE_ROWS = 40960  # positions in the rotation table
IMAGE = 37          # width of the images, in tokens


def _case(name, op, **kw):
    base = {"B": 1, "T": 1, "ragged": False, "Hq": 32, "Hkv": 8, "dk": 128, "dv": 128, "dtype": "bf16",
            "cache": "bf16" if op in ("axes", "weigh", "evict") else "blocks", "page": 64, "block": 0, "len_min": 1,
            "len_max": 1, "window": 0, "pairs": False, "axes": 3 if op == "axes" else 0, "dealt": False, "keep": 0,
            "recent": 0}
    return {"name": name, "op": op, **base, **kw}


def listed():
    return [
        # One stream generating text after an image: the smallest call, all latency.
        _case("axes_b1", "axes", len_min=4095, len_max=4095),
        # Four prompts of images and text entering an empty cache, the axes dealt to the pairs in turn.
        _case("axes_prompt_b4", "axes", B=4, T=5000, dealt=True, len_min=0, len_max=0),
        # Drafts of 48 sequences into a latent cache, time and place of a token on two axes.
        _case("axes_latent_b48", "axes", B=48, T=16, ragged=True, Hkv=1, dk=576, dv=512, pairs=True, axes=2,
              len_min=511, len_max=4000),
        # One stream generating: one token joins a block that holds earlier ones.
        _case("append_b1", "append", block=64, len_min=4093, len_max=4093),
        # A speculative round of 64 sequences, 0 to 7 drafts each.
        _case("append_drafts_b64", "append", B=64, T=7, ragged=True, page=128, block=32, len_min=100, len_max=8000),
        # Eight prompts of 8192 tokens entering an empty cache.
        _case("append_prompt_b8", "append", B=8, T=8192, block=64, len_min=0, len_max=0),
        # One stream with a long context.
        _case("attend_b1_long", "attend", block=64, len_min=131070, len_max=131070),
        # A speculative round: 0 to 4 drafts each of 64 sequences with contexts from 60 to 8191 tokens.
        _case("attend_drafts_b64", "attend", B=64, T=4, ragged=True, page=128, block=16, len_min=60, len_max=8191),
        # A decode step's weights, 64 sequences.
        _case("weigh_b64", "weigh", B=64, len_min=60, len_max=8191),
        # The last 32 tokens of four prompts say what of these is kept, an 8-bit cache.
        _case("weigh_prompt_b4", "weigh", B=4, T=32, cache="blocks", block=64, len_min=7001, len_max=30000),
        # One long context cut to a fifth.
        _case("evict_b1_long", "evict", len_min=100001, len_max=100001, keep=20000, recent=500),
        # A serving batch with a budget of 2000 tokens, an 8-bit cache; the shorter sequences stay as they are.
        _case("evict_b64", "evict", B=64, cache="blocks", block=64, len_min=500, len_max=8191, keep=2000, recent=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["axes", "append", "attend", "weigh", "evict"])
        form = {"axes": ["bf16", "bf16", "e4m3", "f32", "latent"], "append": ["blocks"], "attend": ["blocks"],
                "weigh": ["bf16", "bf16", "e4m3", "f32", "blocks"],
                "evict": ["bf16", "bf16", "e4m3", "f32", "blocks", "latent"]}[op]
        form = rng.choice(form)
        B, page = _log_int(rng, 1, 64), rng.choice([16, 32, 64, 128, 256])
        c = {"op": op, "B": B, "ragged": rng.random() < 0.5, "dtype": "f32" if form == "f32" else "bf16",
             "cache": "bf16" if form == "latent" else form, "page": page, "block": 0, "window": 0,
             "pairs": rng.random() < 0.3, "axes": 0, "dealt": rng.random() < 0.5, "keep": 0, "recent": 0}
        if form == "blocks":
            c["block"] = rng.choice([x for x in (16, 32, 64, 128, 256) if x <= page])
        if form == "latent":
            c |= {"Hq": rng.choice([8, 16, 32, 64]), "Hkv": 1, "dk": 576, "dv": 512}
        else:
            Hkv, d = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128])
            c |= {"Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), "Hkv": Hkv, "dk": d, "dv": d}
            if c["Hq"] > 64:
                continue
        if op in ("axes", "append"):
            c["T"] = rng.choice([1, rng.randint(2, 16), _log_int(rng, 17, 8192)])
            c["axes"] = rng.randint(2, 4) if op == "axes" else rng.choice([0, 0, 3])
            top = _log_int(rng, 1, 16000)
            c["len_min"], c["len_max"] = _log_int(rng, 1, top) - 1, top
        else:
            c["T"] = {"attend": rng.choice([1, 1, rng.randint(2, 8)]), "weigh": rng.choice([1, rng.randint(2, 64)]),
                      "evict": 1}[op]
            top = _log_int(rng, 16, 131000 if B <= 2 else 16000)
            c["len_min"], c["len_max"] = _log_int(rng, 1, top), top
            if op != "evict" and rng.random() < 0.25:
                c["window"] = _log_int(rng, 16, 4096)
            if op == "evict":
                c["keep"] = _log_int(rng, 1, top)
                c["recent"] = rng.choice([0, c["keep"], rng.randint(0, c["keep"]), rng.randint(0, c["keep"]) // 8])
        w = work(c)
        seqs = _spread(c)
        if op == "evict" and all(n <= c["keep"] for n, _ in seqs):
            continue
        if sum(n for _, n in seqs) and w["bytes"] <= 0.9e9 and w["flops"] <= 0.3e11:
            return {k: c[k] for k in sorted(c)}


# ---------------------------------------------------------------- what both forms are given

def _latent(case):
    return case["dk"] != case["dv"]


def _spread(case):
    """Tokens already cached and new tokens of each sequence: a spread that the case alone sets."""
    B, T, lo, hi = case["B"], case["T"], math.log(case["len_min"] + 1), math.log(case["len_max"] + 1)
    new = [T if not case["ragged"] or (T > 16 and b == 0) else (b * 5 + 3) % (min(T, 16) + 1) for b in range(B)]
    return [(int(round(math.exp(lo + (hi - lo) * b / max(B - 1, 1)))) - 1, n) for b, n in enumerate(new)]


def _first(case, p):
    """The first cached token that a query at place p sees."""
    return max(0, p + 1 - case["window"]) if case["window"] else 0


def work(case):
    es = {"bf16": 2, "f32": 4, "e4m3": 1, "blocks": 1}
    e_in, e_c = es[case["dtype"]], es[case["cache"]]
    Hq, Hkv, dk, dv = case["Hq"], case["Hkv"], case["dk"], case["dv"]
    row = dk if _latent(case) else dk + dv
    scales = 8 / case["block"] if case["block"] else 0  # bytes of a token and head
    seqs = _spread(case)
    N = sum(n for _, n in seqs)
    if case["op"] in ("axes", "append"):
        rot = _rotation(case)[1]
        return {"bytes": N * (2 * Hq * dk * e_in + Hkv * (row * (e_in + e_c) + scales) + 4 * rot + 8 * case["axes"]),
                "flops": N * (Hq + Hkv) * rot * 3}
    if case["op"] == "evict":
        long = [p for p, _ in seqs if p > case["keep"]]
        moved = case["keep"] * len(long)
        stride = -(-max(p for p, _ in seqs) // case["page"]) * case["page"]
        return {"bytes": Hkv * (sum(p for p, _ in seqs) * 4 + moved * (2 * row * e_c + 2 * scales + 4)
                                + case["B"] * stride * 4), "flops": 0}
    tokens = pairs = 0
    for p0, n in seqs:
        tokens += p0 + n - _first(case, p0) if n else 0
        pairs += sum(p0 + i + 1 - _first(case, p0 + i) for i in range(n))
    if case["op"] == "weigh":
        return {"bytes": tokens * Hkv * (dk * e_c + scales / 2 + 8) + N * Hq * (dk * e_in + 4),
                "flops": 2 * pairs * Hq * dk}
    return {"bytes": tokens * Hkv * (row * e_c + scales) + N * Hq * ((dk + dv) * e_in + 4),
            "flops": 2 * pairs * Hq * (dk + dv)}


def _rotation(case):
    """Where a head is rotated: (first value, how many)."""
    return (case["dv"], case["dk"] - case["dv"]) if _latent(case) else (0, case["dk"])


def _sections(case):
    """Pairs of each axis: somewhat fewer on the first."""
    half, A = _rotation(case)[1] // 2, case["axes"]
    each = (half + A - 1) // A
    return [half - each * (A - 1)] + [each] * (A - 1)


def _axis_of(case):
    """The axis of each pair: section after section, or dealt in turn while the sections last."""
    left = _sections(case)
    if not case["dealt"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    return [a for i in range(max(left)) for a, n in enumerate(left) if i < n]


def _axis_positions(seqs, axes):
    """Positions of each axis [axes][N]: text counts up all axes alike, an image runs over its rows and columns."""
    def of(p0, n):
        i = np.arange(n)
        j, base = i - n // 4, p0 // 2 + n // 8
        image = (i >= n // 4) & (i < n - n // 4) & (n > 4)
        axis = [base + 0 * j, base + j // IMAGE, base + j % IMAGE, base + j % IMAGE]
        return np.stack([np.where(image, axis[a], (p0 + i) // 2) for a in range(axes)])

    return np.concatenate([of(*x) for x in seqs], 1).astype(np.int64)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    rng = random.Random(seed)
    op, seqs = case["op"], _spread(case)
    rng.shuffle(seqs)
    if op == "evict":
        seqs = [(p, 0) for p, _ in seqs]
    B, T, Hq, Hkv, dk, dv, page, block = (case[k] for k in ("B", "T", "Hq", "Hkv", "dk", "dv", "page", "block"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ct = {"bf16": torch.bfloat16, "f32": torch.float32}.get(case["cache"], torch.float8_e4m3fn)
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    N = starts[-1]
    need = [-(-(p + n) // page) for p, n in seqs]
    moved = [b for b, (p, _) in enumerate(seqs) if op == "evict" and p > case["keep"]]
    dst = -(-case["keep"] // page)
    n_pages, max_pages = sum(need) + dst * len(moved) + 3, max(max(need), 1)
    ids = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    table, at = np.zeros((B, max_pages), dtype=np.int32), 0
    for b, k in enumerate(need):
        table[b, :k], at = ids[at:at + k], at + k

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=g, dtype=dt)

    def pages(width):
        x = torch.randn((n_pages, Hkv, page, width), device=DEV, generator=g,
                        dtype=torch.float32 if ct == torch.float32 else torch.bfloat16)
        return (x * 64).to(ct) if ct == torch.float8_e4m3fn else x.to(ct)

    def block_scales():
        e = torch.randint(-8, -4, (n_pages, Hkv, page // block), device=DEV, generator=g)
        return torch.ldexp(torch.ones((), device=DEV), e)

    s = {"case": case, "N": N, "k_pages": pages(dk), "v_pages": None if _latent(case) else pages(dv),
         "table": torch.from_numpy(table).to(DEV),
         "pos": torch.tensor([p for p, _ in seqs], dtype=torch.int64, device=DEV),
         "tok_start": torch.tensor(starts, dtype=torch.int32, device=DEV), "k_scale": None, "v_scale": None,
         "axis_pos": None,
         # Sequences whose first new token joins earlier ones in its block.
         "joins": torch.tensor([b for b, (p, n) in enumerate(seqs) if block and n and p % block], dtype=torch.int64,
                               device=DEV)}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.01 * (1 + torch.rand((Hkv,), device=DEV, generator=g))
        s["v_scale"] = 0.01 * (1 + torch.rand((Hkv,), device=DEV, generator=g))
    elif case["cache"] == "blocks":
        s["k_scale"], s["v_scale"] = block_scales(), block_scales()
    if op != "evict":
        s["q"] = normal(N, Hq, dk)
    if op in ("axes", "append"):
        s["k"] = normal(N, Hkv, dk)
        s["v"] = None if _latent(case) else normal(N, Hkv, dv)
        first, width = _rotation(case)
        inv = 10000.0 ** (-torch.arange(0, width, 2, device=DEV, dtype=torch.float64) / width)
        ang = torch.arange(TABLE_ROWS, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        if case["axes"]:
            s["axis_pos"] = torch.from_numpy(_axis_positions(seqs, case["axes"])).to(DEV)
            s["axis_of"] = torch.tensor(_axis_of(case), device=DEV)
    if op == "weigh":
        s["lse"] = torch.zeros((N, Hq), device=DEV)
        b, i = _rows(s)
        s["lse"] = torch.logsumexp(_scores(s), -1).transpose(1, 2).reshape(B, T, Hq)[b, i]
    if op in ("weigh", "evict"):
        s["weights"] = torch.randn((B, Hkv, max_pages * page), device=DEV, generator=g).mul_(2).exp_()
        s["weights"][torch.rand(s["weights"].shape, device=DEV, generator=g) < 0.05] = 0
        s["weights"] *= 1e-3  # of the size of what a call adds
    if op == "evict":
        keep = case["keep"]
        dst_table = np.zeros((B, dst), dtype=np.int32)
        for b in moved:
            dst_table[b], at = ids[at:at + dst], at + dst
        s |= {"moved": torch.tensor(moved, dtype=torch.int64, device=DEV), "dst_table": torch.from_numpy(dst_table).to(DEV),
              "kept": torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV),
              "new_pos": torch.empty(B, dtype=torch.int64, device=DEV), "new_weights": torch.empty_like(s["weights"])}
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The library's call, checked once as a serving loop does."""
    import recurrent_state_amd as kda
    case, err = s["case"], torch.zeros(1, dtype=torch.int32, device=DEV)
    pool = kda.PagePool.from_tensors(s["k_pages"], s["v_pages"], dv=case["dv"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"], scale_block=case["block"])
    rows = {"tok_start": s["tok_start"], "T": case["T"]}
    if case["op"] in ("axes", "append"):
        s["q_out"] = torch.empty_like(s["q"])
        if case["axes"]:
            rows |= {"axis_pos": s["axis_pos"],
                     "axis_of": kda.rotation_axes(_sections(case), interleaved=case["dealt"])}
        return kda.KvAppendPlan(pool, s["table"], s["pos"], s["k"], s["v"], err, q=s["q"], q_out=s["q_out"],
                                cos_sin=s["cos_sin"], rot_start=_rotation(case)[0], rot_pairs=case["pairs"], **rows)
    if case["op"] == "evict":
        return kda.KvEvictPlan(pool, s["table"], s["pos"], s["weights"], s["dst_table"], s["new_pos"],
                               s["new_weights"], s["kept"], err, recent=case["recent"])
    rows |= {"scale": case["dk"] ** -0.5, "window": case["window"]}
    if case["op"] == "weigh":
        return kda.AttnWeightsPlan(pool, s["table"], s["pos"], s["q"], s["lse"], s["weights"], err, **rows)
    s["o"] = torch.empty((s["N"], case["Hq"], case["dv"]), device=DEV, dtype=s["q"].dtype)
    s["lse"] = torch.empty((s["N"], case["Hq"]), device=DEV, dtype=torch.float32)
    ws = kda.attn_workspace(pool, s["table"], Hq=case["Hq"], T=case["T"])
    return kda.AttnDecodePlan(pool, s["table"], s["pos"], s["q"], s["o"], ws, err, lse=s["lse"], **rows)


def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        if op in ("axes", "append"):
            return _cache(s, q=s["q_out"])
        if op == "weigh":
            return {"weights": s["weights"]}
        return _evicted(s) if op == "evict" else {"o": s["o"], "lse": s["lse"]}
    return {"axes": _append, "append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[op](s)


def _cache(s, **more):
    """The pages, and what scales them where the call sets it."""
    out = {"k_pages": s["k_pages"], **more}
    if s["v_pages"] is not None:
        out["v_pages"] = s["v_pages"]
    if s["case"]["block"]:
        out |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out


def _evicted(s):
    return _cache(s, kept=s["kept"], new_pos=s["new_pos"], new_weights=s["new_weights"])


# ---------------------------------------------------------------- the plain forms

def _rows(s):
    """For each token row: its sequence and its place among the sequence's new tokens."""
    r = torch.arange(s["N"], device=DEV)
    b = torch.searchsorted(s["tok_start"].long(), r, right=True) - 1
    return b, r - s["tok_start"].long()[b]


def _rotate(x, cos, sin, first, pairs):
    """x in 32 bits with its values first .. first + 2 * cos.shape[-1] - 1 rotated."""
    half = cos.shape[-1]
    y = x.clone()
    if pairs:
        i, j = slice(first, first + 2 * half, 2), slice(first + 1, first + 2 * half, 2)
    else:
        i, j = slice(first, first + half), slice(first + half, first + 2 * half)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    return y


def _bits(pages):
    """8-bit pages as bytes, which indexing takes."""
    return pages.view(torch.uint8) if pages.element_size() == 1 else pages


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _block_scale(m):
    """The smallest power of two, 2^-64 or more, by which values up to m divide to at most 448."""
    part, e = torch.frexp(m)  # m = part 2^e, 448 = 0.875 * 2^9
    e = e - 9 + (part > 0.875)
    return torch.ldexp(torch.ones_like(m), torch.where(m > 0, e, -64).clamp(min=-64))


def _append(s):
    case = s["case"]
    b, i = _rows(s)
    p = s["pos"][b] + i
    page, slot = s["table"][b, p // case["page"]].long(), p % case["page"]
    if s["axis_pos"] is None:
        cs = s["cos_sin"][p]
    else:
        lead = torch.arange(len(s["axis_of"]), device=DEV)
        at = s["axis_pos"][s["axis_of"]].T
        cs = torch.cat([s["cos_sin"][at, lead], s["cos_sin"][at, len(lead) + lead]], 1)
    cos, sin = cs[:, None].chunk(2, -1)
    first = _rotation(case)[0]
    _store(s, "k", _rotate(s["k"].float(), cos, sin, first, case["pairs"]), b, page, slot)
    if s["v"] is not None:
        _store(s, "v", s["v"].float(), b, page, slot)
    return _cache(s, q=_rotate(s["q"].float(), cos, sin, first, case["pairs"]).to(s["q"].dtype))


def _store(s, name, x, b, page, slot):
    """New rows x to their places; where blocks have scales, with the scales that they then need."""
    case, pages, scale = s["case"], s[name + "_pages"], s[name + "_scale"]
    if case["block"]:
        x = _store_scales(s, pages, scale, x, b, page, slot)
    elif scale is not None:
        x = x / scale[:, None]
    _bits(pages)[page, :, slot] = _bits(_e4m3(x) if pages.element_size() == 1 else x.to(pages.dtype))


def _store_scales(s, pages, scale, x, b, page, slot):
    """x over its blocks' new scales, which are written, and a block's earlier tokens stored anew."""
    Hkv, block = s["case"]["Hkv"], s["case"]["block"]
    per, spans = s["case"]["page"] // block, s["tok_start"].long()
    old = scale.transpose(1, 2).reshape(-1, Hkv)
    g = page * per + slot // block
    top = torch.zeros_like(old).scatter_reduce_(0, g[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
    new = _block_scale(top)
    # Only the block of a sequence's first new token can hold earlier ones.
    lead = spans[:-1][s["joins"]]
    begun = g[lead]
    new[begun] = torch.maximum(new[begun], old[begun])
    hit = torch.zeros(len(old), dtype=torch.bool, device=DEV).index_fill_(0, g, True)
    new = torch.where(hit[:, None], new, old)
    j = torch.arange(block, device=DEV)
    at = (begun[:, None] // per, slice(None), begun[:, None] % per * block + j)  # [joins][block][heads][width]
    was = _bits(pages)[at]
    now = _bits(_e4m3(was.view(pages.dtype).float() * (old / new)[begun][:, None, :, None]))
    _bits(pages)[at] = torch.where((j < (slot % block)[lead][:, None])[..., None, None], now, was)
    scale.copy_(new.view(-1, per, Hkv).transpose(1, 2))
    return x / new[g][:, :, None]


def _gathered(s, name):
    """[B][kv heads][places][width] in 32 bits."""
    pages, scale, table = s[name + "_pages"], s[name + "_scale"], s["table"]
    x = _bits(pages)[table].view(pages.dtype).float()
    if s["case"]["block"]:
        x = (x.unflatten(3, (-1, s["case"]["block"])) * scale[table][..., None, None]).flatten(3, 4)
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None or s["case"]["block"] else x * scale[:, None, None]


def _scores(s):
    """[B][kv heads][T][group][places], -inf where a row does not see a token."""
    case = s["case"]
    B, T, Hq, Hkv, dk = (case[k] for k in ("B", "T", "Hq", "Hkv", "dk"))
    t = torch.arange(T, device=DEV)
    row = (s["tok_start"][:-1].long()[:, None] + t).clamp(max=s["N"] - 1)
    q = s["q"].float()[row].view(B, T, Hkv, Hq // Hkv, dk).transpose(1, 2).reshape(B, Hkv, -1, dk)
    K = _gathered(s, "k")
    x = (q @ K.transpose(-1, -2)).view(B, Hkv, T, Hq // Hkv, -1) * dk ** -0.5
    p, j = (s["pos"][:, None] + t)[..., None], torch.arange(K.shape[2], device=DEV)
    hidden = j > p
    if case["window"]:
        hidden |= j <= p - case["window"]
    return x.masked_fill(hidden[:, None, :, None, :], -math.inf)


def _attend(s):
    case = s["case"]
    B, T, Hq, Hkv, dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "dv"))
    b, i = _rows(s)
    x = _scores(s)
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    o = ((e / total).view(B, Hkv, -1, x.shape[-1]) @ _gathered(s, "v")).view(B, Hkv, T, Hq // Hkv, dv)
    o = o.transpose(1, 2).reshape(B, T, Hq, dv)[b, i].to(s["q"].dtype)
    return {"o": o, "lse": (m + total.log()).squeeze(-1).transpose(1, 2).reshape(B, T, Hq)[b, i]}


def _weigh(s):
    case, starts = s["case"], s["tok_start"].long()
    B, T, Hq, Hkv = (case[k] for k in ("B", "T", "Hq", "Hkv"))
    t = torch.arange(T, device=DEV)
    n = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + t).clamp(max=s["N"] - 1)
    lse = s["lse"][row].view(B, T, Hkv, -1).transpose(1, 2)[..., None]
    e = (_scores(s) - lse).exp().masked_fill((t >= n[:, None])[:, None, :, None, None], 0)
    j, pos = torch.arange(e.shape[-1], device=DEV), s["pos"][:, None]
    sums = torch.where(j < pos, 1.0, 0.0)[:, None] * s["weights"] + e.sum((2, 3))
    seen = (n[:, None] > 0) & (j < pos + n[:, None])
    if case["window"]:
        seen &= j > pos - case["window"]
    s["weights"].copy_(torch.where(seen[:, None], sums, s["weights"]))
    return {"weights": s["weights"]}


def _evict(s):
    case, moved = s["case"], s["moved"]
    keep, page = case["keep"], case["page"]
    L, j = s["pos"][:, None, None], torch.arange(s["weights"].shape[-1], device=DEV)
    rank = s["weights"].masked_fill(j >= L - case["recent"], math.inf).masked_fill(j >= L, -math.inf)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.nn.functional.pad(kept, (0, max(0, keep - kept.shape[-1])))[..., :keep].sort(-1).values
    shorter = L <= keep
    s["kept"].copy_(torch.where(shorter, -1, kept))
    s["new_pos"].copy_(s["pos"].clamp(max=keep))
    stays = torch.where(j < L, s["weights"], 0)
    goes = torch.nn.functional.pad(s["weights"].gather(-1, kept), (0, max(0, len(j) - keep)))[..., :len(j)]
    s["new_weights"].copy_(torch.where(shorter, stays, goes))
    kept, i = kept[moved], torch.arange(keep, device=DEV)  # [moved][kv heads][keep]
    h = torch.arange(case["Hkv"], device=DEV)[:, None]
    src = s["table"][moved[:, None, None], kept // page].long(), h, kept % page
    to = s["dst_table"][moved][:, i // page].long()[:, None], h, i % page
    _move(s, "k", src, to)
    if s["v_pages"] is not None:
        _move(s, "v", src, to)
    return _evicted(s)


def _move(s, name, src, to):
    """Rows from places to places; where blocks have scales, with the scales that they need there."""
    pages, scale, block = s[name + "_pages"], s[name + "_scale"], s["case"]["block"]
    rows = _bits(pages)[src]
    if block:
        x = rows.view(pages.dtype).float() * scale[src[0], src[1], src[2] // block][..., None]
        n = x.shape[2]
        top = torch.nn.functional.pad(x.abs().amax(-1), (0, -n % block)).unflatten(-1, (-1, block)).amax(-1)
        new = _block_scale(top)
        first = slice(0, n, block)
        scale[to[0][..., first], to[1], to[2][first] // block] = new
        rows = _bits(_e4m3(x / new.repeat_interleave(block, -1)[..., :n, None]))
    _bits(pages)[to] = rows


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"axes": _exact_append, "append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](s)


def _places(s, b, first, past):
    """(page, slot) of the places first .. past - 1 of sequence b."""
    at = torch.arange(first, past, device=DEV)
    return s["table"].long()[b, at // s["case"]["page"]], at % s["case"]["page"]


def _fitting(m):
    """log2 of _block_scale's answer, from logarithms."""
    e = torch.ceil(torch.log2(m.double().clamp(min=1e-300) / 448))
    return torch.where(m > 0, e, -64.0).clamp(min=-64)


def _exact_append(s):
    case = s["case"]
    Hkv, block = case["Hkv"], case["block"]
    if s["N"] * case["Hq"] * case["dk"] > 1 << 28:
        return None
    starts, pos = s["tok_start"].tolist(), s["pos"].tolist()
    first, width = _rotation(case)
    lead = torch.arange(width // 2, device=DEV)
    i, j = (first + 2 * lead, first + 2 * lead + 1) if case["pairs"] else (first + lead, first + width // 2 + lead)
    out = {"q": s["q"].double(), "k_pages": s["k_pages"].double()}
    if s["v"] is not None:
        out["v_pages"] = s["v_pages"].double()
    if block:
        out |= {"k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}

    def turn(x, b):
        r = torch.arange(starts[b], starts[b + 1], device=DEV)
        at = (torch.arange(pos[b], pos[b] + len(r), device=DEV)[:, None].expand(-1, len(lead))
              if s["axis_pos"] is None else s["axis_pos"][s["axis_of"]][:, r].T)
        c, si = s["cos_sin"][at, lead].double()[:, None], s["cos_sin"][at, len(lead) + lead].double()[:, None]
        z = torch.complex(x[..., i], x[..., j]) * torch.complex(c, si)
        y = x.clone()
        y[..., i], y[..., j] = z.real, z.imag
        return y

    def put(name, x, b):
        pages, n = out[name + "_pages"], len(x)
        pg, sl = _places(s, b, pos[b], pos[b] + n)
        if not block:
            scale = s[name + "_scale"]
            pages[pg, :, sl] = x if scale is None else (x / scale.double()[:, None]).clamp(-448, 448)
            return
        scales, at = out[name + "_scale"], pos[b]
        while at < pos[b] + n:
            past = min(pos[b] + n, (at // block + 1) * block)
            new, page, k = x[at - pos[b]:past - pos[b]], int(pg[at - pos[b]]), int(sl[at - pos[b]]) // block
            held = int(sl[at - pos[b]]) % block
            e = _fitting(new.abs().amax((0, 2)))
            if held:
                e = torch.maximum(e, torch.log2(scales[page, :, k]))
                pages[page, :, k * block:k * block + held] *= (scales[page, :, k] / 2.0 ** e)[:, None, None]
            scales[page, :, k] = 2.0 ** e
            pages[page, :, k * block + held:k * block + held + past - at] = \
                (new / (2.0 ** e)[:, None]).clamp(-448, 448).transpose(0, 1)
            at = past

    if block and s["N"] / block + case["B"] > 4000:
        return None
    for b in range(case["B"]):
        r = slice(starts[b], starts[b + 1])
        if r.stop > r.start:
            out["q"][r] = turn(s["q"][r].double(), b)
            put("k", turn(s["k"][r].double(), b), b)
            if s["v"] is not None:
                put("v", s["v"][r].double(), b)
    return out


def _cached(s, name, b, past):
    """[kv heads][past][width] of sequence b's places in 64 bits."""
    pages, scale = s[name + "_pages"], s[name + "_scale"]
    pg, sl = _places(s, b, 0, past)
    x = _bits(pages)[pg, :, sl].view(pages.dtype).double().transpose(0, 1)
    if s["case"]["block"]:
        return x * scale[pg, :, sl // s["case"]["block"]].double().T[..., None]
    return x if scale is None else x * scale.double()[:, None, None]


def _exact_scores(s, k, b, r, p):
    """(first token that the row sees, its scores [kv heads][group][tokens])."""
    case, lo = s["case"], _first(s["case"], p)
    z = torch.matmul(s["q"][r].double().view(case["Hkv"], -1, case["dk"]), k[:, lo:p + 1].transpose(1, 2).contiguous())
    return lo, z / math.sqrt(case["dk"])


def _exact_attend(s):
    case, starts, pos = s["case"], s["tok_start"].tolist(), s["pos"].tolist()
    o = torch.zeros((s["N"], case["Hq"], case["dv"]), dtype=torch.float64, device=DEV)
    lse = torch.full((s["N"], case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        past = pos[b] + starts[b + 1] - starts[b]
        k, v = _cached(s, "k", b, past), _cached(s, "v", b, past)
        for r in range(starts[b], starts[b + 1]):
            p = pos[b] + r - starts[b]
            lo, z = _exact_scores(s, k, b, r, p)
            lse[r] = torch.logsumexp(z, -1).flatten()
            o[r] = torch.matmul(torch.softmax(z, -1), v[:, lo:p + 1].contiguous()).view(case["Hq"], -1)
    return {"o": o, "lse": lse}


def _exact_weigh(s):
    case, starts, pos = s["case"], s["tok_start"].tolist(), s["pos"].tolist()
    w = s["weights"].double()
    for b in range(case["B"]):
        k = _cached(s, "k", b, pos[b] + starts[b + 1] - starts[b])
        w[b, :, pos[b]:pos[b] + starts[b + 1] - starts[b]] = 0
        for r in range(starts[b], starts[b + 1]):
            p = pos[b] + r - starts[b]
            lo, z = _exact_scores(s, k, b, r, p)
            w[b, :, lo:p + 1] += torch.exp(z - s["lse"][r].double().view(case["Hkv"], -1, 1)).sum(1)
    return {"weights": w}


def _exact_evict(s):
    case, pos = s["case"], s["pos"].tolist()
    keep, block, page = case["keep"], case["block"], case["page"]
    names = ["k", "v"] if s["v_pages"] is not None else ["k"]
    w, dst = s["weights"].cpu().numpy(), s["dst_table"].long()
    out = {n + "_pages": s[n + "_pages"].double() for n in names}
    if block:
        out |= {n + "_scale": s[n + "_scale"].double() for n in names}
    out |= {"kept": torch.full_like(s["kept"], -1), "new_pos": s["pos"].clamp(max=keep),
            "new_weights": torch.zeros_like(s["weights"], dtype=torch.float64)}
    if case["B"] * case["Hkv"] > 600 or keep * case["Hkv"] * len(s["moved"]) * case["dk"] > 1 << 28:
        return None
    for b in range(case["B"]):
        out["new_weights"][b, :, :pos[b]] = s["weights"][b, :, :pos[b]].double()
        if pos[b] <= keep:
            continue
        out["new_weights"][b] = 0
        for h in range(case["Hkv"]):
            cut = pos[b] - case["recent"]
            best = np.argsort(-w[b, h, :cut].astype(np.float64), kind="stable")[:keep - case["recent"]]
            kept = torch.from_numpy(np.concatenate([np.sort(best), np.arange(cut, pos[b])])).to(DEV)
            out["kept"][b, h] = kept.int()
            out["new_weights"][b, h, :keep] = s["weights"][b, h, kept].double()
            src = s["table"].long()[b, kept // page]
            i = torch.arange(keep, device=DEV)
            for n in names:
                x = _bits(s[n + "_pages"])[src, h, kept % page].view(s[n + "_pages"].dtype).double()
                if block:
                    x = x * s[n + "_scale"][src, h, kept % page // block].double()[:, None]
                    e = torch.stack([_fitting(c.abs().amax()) for c in x.split(block)])
                    out[n + "_scale"][dst[b, i[::block] // page], h, i[::block] % page // block] = 2.0 ** e
                    x = x / (2.0 ** e).repeat_interleave(block)[:keep, None]
                out[n + "_pages"][dst[b, i // page], h, i % page] = x
    return out
