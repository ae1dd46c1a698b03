"""The operators on the paged attention cache: what is timed, and their plain forms.

A hybrid stack alternates recurrent-state layers with attention layers.  The attention layers'
cache grows with the sequence and lives in pages; two operators serve it:

  append   new keys and values go to their pages, rotated by their positions on the way; the
           queries of the same tokens are rotated in the same pass
  attend   the new tokens' queries read the cache: softmax attention over all cached tokens (or
           the last `window` of them) up to and including their own position

Layouts: queries, keys and values are packed token rows [N][heads][width], sequence b owning rows
tok_start[b] .. tok_start[b + 1] - 1 at positions pos[b], pos[b] + 1, ...; the cache holds
[pages][kv heads][page size][width]; table[b][i] is the page with tokens i * page size and on.
A latent cache has one row per token that all query heads share: the row is the key, its first
`dv` values are the value.  An 8-bit cache holds e4m3 values of x / scale, one scale per kv head.

With `own` false, run() computes the plain forms from elementary torch operations in 32 bits;
with `own` true it makes the library's calls.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TABLE_ROWS = 132096  # positions in the rotation table: the longest sequence and its new tokens


def _case(name, op, **kw):
    base = {"B": 1, "T": 1, "ragged": False, "Hq": 32, "Hkv": 8, "dk": 128, "dv": 128, "latent": False,
            "dtype": "bf16", "cache": "bf16", "page": 64, "len_min": 1, "len_max": 1, "window": 0, "pairs": False}
    return {"name": name, "op": op, **base, **kw}


def listed():
    return [
        # One stream generating: the smallest append, all latency.
        _case("append_b1", "append", len_min=4095, len_max=4095),
        # A speculative round of 64 sequences, 0 to 7 drafts each, into an 8-bit cache.
        _case("append_drafts_b64_e4m3", "append", B=64, T=7, ragged=True, cache="e4m3", len_min=100, len_max=8000),
        # Eight prompts of 8192 tokens entering an empty cache.
        _case("append_prompt_b8", "append", B=8, T=8192, len_min=0, len_max=0),
        # Four drafts each of 64 sequences into a latent cache: 64 of a row's 576 values are rotated.
        _case("append_latent_b64", "append", B=64, T=4, Hkv=1, dk=576, dv=512, latent=True, pairs=True,
              len_min=511, len_max=4000),
        # One stream with a short context: few pages, all latency.
        _case("attend_b1_short", "attend", len_min=1020, len_max=1020),
        # One stream with a long context: the cache is split over the whole chip and joined.
        _case("attend_b1_long", "attend", len_min=131070, len_max=131070),
        # A serving batch with contexts from 60 to 8191 tokens.
        _case("attend_b64", "attend", B=64, len_min=60, len_max=8191),
        # A speculative round: 0 to 4 drafts each of 16 sequences, 8 query heads to a kv head.
        _case("attend_drafts_b16", "attend", B=16, T=4, ragged=True, Hkv=4, page=16, len_min=1001, len_max=4500),
        # Long contexts in an 8-bit cache.
        _case("attend_b32_e4m3", "attend", B=32, cache="e4m3", page=128, len_min=4000, len_max=16001),
        # Heads of 64 in 32 bits, one kv head to each query head, the last 256 tokens only.
        _case("attend_window_f32", "attend", B=8, Hq=16, Hkv=16, dk=64, dv=64, dtype="f32", cache="f32", page=32,
              len_min=100, len_max=2000, window=256),
        # One stream over a latent cache.
        _case("attend_latent_b1", "attend", Hkv=1, dk=576, dv=512, latent=True, len_min=8190, len_max=8190),
        # Drafts over a latent cache: 128 query rows share each cached row.
        _case("attend_latent_b64", "attend", B=64, T=4, Hkv=1, dk=576, dv=512, latent=True, len_min=500,
              len_max=4090),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend"])
        form = rng.choice(["bf16", "bf16", "e4m3", "f32", "latent"])
        B = _log_int(rng, 1, 64)
        c = {"op": op, "B": B, "ragged": rng.random() < 0.5, "latent": form == "latent",
             "dtype": "f32" if form == "f32" else "bf16", "cache": form if form in ("e4m3", "f32") else "bf16",
             "page": rng.choice([16, 32, 64, 128, 256]), "window": 0, "pairs": rng.random() < 0.3}
        if form == "latent":
            c |= {"Hq": rng.choice([8, 16, 32, 64]), "Hkv": 1, "dk": 576, "dv": 512}
        else:
            Hkv, d = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128])
            c |= {"Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), "Hkv": Hkv, "dk": d, "dv": d}
            if c["Hq"] > 64:
                continue
        if op == "append":
            c["T"] = rng.choice([1, rng.randint(2, 16), _log_int(rng, 17, 8192)])
            top = _log_int(rng, 1, 16000)
            c["len_min"], c["len_max"] = _log_int(rng, 1, top) - 1, top
        else:
            c["T"] = rng.choice([1, 1, rng.randint(2, 8)])
            top = _log_int(rng, 16, 131000 if B <= 2 else 16000)
            c["len_min"], c["len_max"] = _log_int(rng, 1, top), top
            if rng.random() < 0.25:
                c["window"] = _log_int(rng, 16, 4096)
        w = work(c)
        if sum(n for _, n in _spread(c)) and w["bytes"] <= 0.9e9 and w["flops"] <= 0.6e11:
            return {k: c[k] for k in sorted(c)}


# ---------------------------------------------------------------- what both forms are given

def _spread(case):
    """Tokens already cached and new tokens of each sequence: a spread that the case alone sets."""
    B, T, lo, hi = case["B"], case["T"], case["len_min"], case["len_max"]
    out = []
    for b in range(B):
        x = 0.0 if B == 1 else b / (B - 1)
        n = T if not case["ragged"] else T if T > 16 and b == 0 else (b * 5 + 3) % (min(T, 16) + 1)
        out.append((int(round(math.exp((1 - x) * math.log(lo + 1) + x * math.log(hi + 1)))) - 1, n))
    return out


def _range(case, p0, n):
    """The cached tokens that some new token of the sequence sees: [first, past the last)."""
    lo = max(0, p0 + 1 - case["window"]) if case["window"] else 0
    return (lo, p0 + n) if n else (0, 0)


def work(case):
    es = {"bf16": 2, "f32": 4, "e4m3": 1}
    e_in, e_c = es[case["dtype"]], es[case["cache"]]
    Hq, Hkv, dk, dv = case["Hq"], case["Hkv"], case["dk"], case["dv"]
    row = dk if case["latent"] else dk + dv
    seqs = _spread(case)
    N = sum(n for _, n in seqs)
    rot = 64 if case["latent"] else dk
    if case["op"] == "append":
        return {"bytes": N * (2 * Hq * dk * e_in + Hkv * row * (e_in + e_c) + 4 * rot),
                "flops": N * (Hq + Hkv) * rot * 3}
    tokens = pairs = 0
    for p0, n in seqs:
        lo, hi = _range(case, p0, n)
        tokens += hi - lo
        pairs += sum(p0 + i + 1 - (max(0, p0 + i + 1 - case["window"]) if case["window"] else 0) for i in range(n))
    return {"bytes": tokens * Hkv * row * e_c + N * Hq * ((dk + dv) * e_in + 4), "flops": 2 * pairs * Hq * (dk + dv)}


def _rotation(case):
    """Where a head is rotated: (first value, how many)."""
    return (case["dv"], case["dk"] - case["dv"]) if case["latent"] else (0, case["dk"])


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    rng = random.Random(seed)
    seqs = _spread(case)
    rng.shuffle(seqs)
    B, T, Hq, Hkv, dk, dv, page = (case[k] for k in ("B", "T", "Hq", "Hkv", "dk", "dv", "page"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ct = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}[case["cache"]]
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    N = starts[-1]
    need = [-(-(p + n) // page) for p, n in seqs]
    n_pages, max_pages = sum(need) + 3, max(max(need), 1)
    ids = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    table, at = np.zeros((B, max_pages), dtype=np.int32), 0
    for b, k in enumerate(need):
        table[b, :k], at = ids[at:at + k], at + k

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=g, dtype=dt)

    def pages(width):
        x = torch.randn((n_pages, Hkv, page, width), device=DEV, generator=g,
                        dtype=torch.float32 if ct == torch.float32 else torch.bfloat16)
        return (x * 8).to(ct) if ct == torch.float8_e4m3fn else x

    s = {"case": case, "N": N, "k_pages": pages(dk), "v_pages": None if case["latent"] else pages(dv),
         "table": torch.from_numpy(table).to(DEV),
         "pos": torch.tensor([p for p, _ in seqs], dtype=torch.int64, device=DEV),
         "tok_start": torch.tensor(starts, dtype=torch.int32, device=DEV), "k_scale": None, "v_scale": None}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.02 * (1 + torch.rand((Hkv,), device=DEV, generator=g))
        s["v_scale"] = 0.02 * (1 + torch.rand((Hkv,), device=DEV, generator=g))
        if case["op"] == "attend":  # pages hold about unit normal values: e4m3 values of x / scale
            s["k_scale"], s["v_scale"] = s["k_scale"] * 4, s["v_scale"] * 4
    s["q"] = normal(N, Hq, dk)
    if case["op"] == "append":
        s["k"] = normal(N, Hkv, dk)
        s["v"] = None if case["latent"] else normal(N, Hkv, dv)
        first, width = _rotation(case)
        inv = 10000.0 ** (-torch.arange(0, width, 2, device=DEV, dtype=torch.float64) / width)
        ang = torch.arange(TABLE_ROWS, device=DEV, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    if own:
        import recurrent_state_amd as kda
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["pool"] = kda.PagePool.from_tensors(s["k_pages"], s["v_pages"], dv=dv, k_scale=s["k_scale"],
                                              v_scale=s["v_scale"])
        if case["op"] == "append":
            s["q_out"] = torch.empty_like(s["q"])
            s["call"] = kda.KvAppendPlan(s["pool"], s["table"], s["pos"], s["k"], s["v"], err, q=s["q"],
                                         q_out=s["q_out"], cos_sin=s["cos_sin"], rot_start=_rotation(case)[0],
                                         rot_pairs=case["pairs"], tok_start=s["tok_start"], T=T)
        else:
            s["o"] = torch.empty((N, Hq, dv), device=DEV, dtype=dt)
            s["lse"] = torch.empty((N, Hq), device=DEV, dtype=torch.float32)
            ws = kda.attn_workspace(s["pool"], s["table"], Hq=Hq, T=T)
            s["call"] = kda.AttnDecodePlan(s["pool"], s["table"], s["pos"], s["q"], s["o"], ws, err, lse=s["lse"],
                                           scale=dk ** -0.5, window=case["window"], tok_start=s["tok_start"], T=T)
    return s


def run(s):
    if own:
        s["call"]()
        if s["case"]["op"] == "append":
            return _appended(s, s["q_out"])
        return {"o": s["o"], "lse": s["lse"]}
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


def _appended(s, q_out):
    out = {"q": q_out, "k_pages": s["k_pages"]}
    return out if s["v_pages"] is None else {**out, "v_pages": s["v_pages"]}


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


def _stored(x, scale, like):
    if scale is None:
        return x.to(like.dtype)
    return (x / scale[:, None]).clamp(-448, 448).to(like.dtype)


def _append(s):
    case = s["case"]
    b, i = _rows(s)
    p = s["pos"][b] + i
    page, slot = s["table"][b, p // case["page"]].long(), p % case["page"]
    cs = s["cos_sin"][p][:, None, :]
    cos, sin = cs.chunk(2, -1)
    first = _rotation(case)[0]
    kr = _stored(_rotate(s["k"].float(), cos, sin, first, case["pairs"]), s["k_scale"], s["k_pages"])
    bytewise = kr.element_size() == 1
    (s["k_pages"].view(torch.uint8) if bytewise else s["k_pages"])[page, :, slot] = kr.view(torch.uint8) if bytewise else kr
    if s["v_pages"] is not None:
        vr = _stored(s["v"].float(), s["v_scale"], s["v_pages"])
        (s["v_pages"].view(torch.uint8) if bytewise else s["v_pages"])[page, :, slot] = vr.view(torch.uint8) if bytewise else vr
    return _appended(s, _rotate(s["q"].float(), cos, sin, first, case["pairs"]).to(s["q"].dtype))


def _gathered(pages, table, scale):
    """[B][kv heads][tokens][width] in 32 bits."""
    x = (pages.view(torch.uint8)[table].view(pages.dtype) if pages.element_size() == 1 else pages[table]).float()
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[:, None, None]


def _attend(s):
    case = s["case"]
    B, T, Hq, Hkv, dk, dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "dk", "dv"))
    b, i = _rows(s)
    t = torch.arange(T, device=DEV)
    row = (s["tok_start"][:-1].long()[:, None] + t).clamp(max=s["N"] - 1)
    q = s["q"].float()[row].view(B, T, Hkv, Hq // Hkv, dk).transpose(1, 2).reshape(B, Hkv, -1, dk)
    K = _gathered(s["k_pages"], s["table"], s["k_scale"])
    V = K[..., :dv] if case["latent"] else _gathered(s["v_pages"], s["table"], s["v_scale"])
    x = (q @ K.transpose(-1, -2)).view(B, Hkv, T, Hq // Hkv, -1) * dk ** -0.5
    p, j = (s["pos"][:, None] + t)[..., None], torch.arange(K.shape[2], device=DEV)
    hidden = j > p
    if case["window"]:
        hidden |= j <= p - case["window"]
    x = x.masked_fill(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    o = ((e / total).view(B, Hkv, -1, K.shape[2]) @ V).view(B, Hkv, T, Hq // Hkv, dv)
    o = o.transpose(1, 2).reshape(B, T, Hq, dv)[b, i].to(s["q"].dtype)
    return {"o": o, "lse": (m + total.log()).squeeze(-1).transpose(1, 2).reshape(B, T, Hq)[b, i]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    starts, pos, table = s["tok_start"].tolist(), s["pos"].tolist(), s["table"].long()
    page, Hkv, dv = case["page"], case["Hkv"], case["dv"]
    of = lambda scale: 1.0 if scale is None else scale.double()[:, None]  # noqa: E731
    if case["op"] == "append":
        if s["N"] * case["Hq"] * case["dk"] > 1 << 29:
            return None
        q_all, k_pages = s["q"].double(), s["k_pages"].double()
        v_pages = None if s["v_pages"] is None else s["v_pages"].double()
        first, width = _rotation(case)
        lead = torch.arange(width // 2, device=DEV)
        i, j = (first + 2 * lead, first + 2 * lead + 1) if case["pairs"] else (first + lead, first + width // 2 + lead)

        def turn(x, at):
            c, si = s["cos_sin"][at].double().view(-1, 1, 2, width // 2).unbind(2)
            z = torch.complex(x[..., i], x[..., j]) * torch.complex(c, si)
            y = x.clone()
            y[..., i], y[..., j] = z.real, z.imag
            return y

        def put(pages, pg, sl, x, scale):
            y = x / of(scale)
            pages[pg, :, sl] = y if scale is None else y.clamp(-448, 448)

        for b in range(case["B"]):
            r0, r1 = starts[b], starts[b + 1]
            at = torch.arange(pos[b], pos[b] + r1 - r0, device=DEV)
            pg, sl = table[b, at // page], at % page
            q_all[r0:r1] = turn(q_all[r0:r1], at)
            put(k_pages, pg, sl, turn(s["k"][r0:r1].double(), at), s["k_scale"])
            if v_pages is not None:
                put(v_pages, pg, sl, s["v"][r0:r1].double(), s["v_scale"])
        out = {"q": q_all, "k_pages": k_pages}
        return out if v_pages is None else {**out, "v_pages": v_pages}
    o = torch.zeros((s["N"], case["Hq"], dv), dtype=torch.float64, device=DEV)
    lse = torch.full((s["N"], case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        if starts[b + 1] == starts[b]:
            continue
        ids = table[b, :-(-(pos[b] + starts[b + 1] - starts[b]) // page)]
        both = [None if x is None else (x.view(torch.uint8)[ids].view(x.dtype) if x.element_size() == 1 else x[ids])
                for x in (s["k_pages"], s["v_pages"])]
        k, v = (None if x is None else x.double().transpose(0, 1).flatten(1, 2) for x in both)
        k = k * (1.0 if s["k_scale"] is None else s["k_scale"].double()[:, None, None])
        v = k[..., :dv] if v is None else v * (1.0 if s["v_scale"] is None else s["v_scale"].double()[:, None, None])
        for r in range(starts[b], starts[b + 1]):
            p = pos[b] + r - starts[b]
            lo = max(0, p + 1 - case["window"]) if case["window"] else 0
            z = torch.matmul(s["q"][r].double().view(Hkv, -1, case["dk"]), k[:, lo:p + 1].transpose(1, 2).contiguous())
            z = z / math.sqrt(case["dk"])
            lse[r] = torch.logsumexp(z, -1).flatten()
            o[r] = torch.matmul(torch.softmax(z, -1), v[:, lo:p + 1].contiguous()).view(-1, dv)
    return {"o": o, "lse": lse}
