"""Measured cases of the serving operators around a 4-bit paged KV cache.

The operators, in the order a decode step calls them:

``norm_rope``  RMS norm of every query and key head and the position rotation,
               in one pass (``sz_qk_norm_rope``).
``append``     K and V rows quantised to 4 bits into the cache's pages, then
               read back as bf16: what a prompt processed in pieces does, so
               that it attends to the same values that later steps will see
               (``sz_cache_append``, ``sz_cache_read``).
``attend``     one query token per sequence over the 4-bit pages, with the
               attention weights added up per cached token where an eviction
               will use them (``sz_cache_attend``).
``evict``      each kv head keeps its `keep` tokens of most accumulated
               weight, the `recent` last positions among them, and the pages
               are compacted in place (``sz_cache_evict``).

Cache format.  A page holds `page_tokens` tokens of every kv head, as
[kv head][cell of 16 tokens].  A cell of head dimension D is
[K codes 8D bytes][V codes 8D][K scales D][V scales D]; channel c of a token
stands for (code - 8) * scale[c // 32], with 4-bit codes 1..15 and bf16 scales.
  K code of token t, channel 32i + 8q + 4h + e: nibble e of 16-bit word
    ((t * 4 + q) * D/32 + i) * 2 + h.
  V code of token 8b + 2q + h, channel 32i + 4g + e: nibble e of 16-bit word
    (((b * 8 + g) * 4 + q) * D/32 + i) * 2 + h.
  scale of token 2p + h, group i: 16-bit word (p * D/32 + i) * 2 + h.
Quantisation of a group of 32 channels: scale = bf16(max|x| / 7), zero when
that is below 2^-126, NaN when the group holds an infinity or a NaN;
code = 8 + round(x / scale), ties to even, clamped to 1..15, and 8 where the
scale is zero or NaN.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CELL = 16
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # One decode step of a batch: 64 sequences, one token each.
        {"name": "norm_rope step 64", "op": "norm_rope", "tokens": 64, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "far": 32768},
        # A whole 8,192-token prompt of the prefill configuration.
        {"name": "norm_rope prompt 8192", "op": "norm_rope", "tokens": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "far": 8192},
        # Packed prompts of odd total length, adjacent pairs, half of the
        # channels rotated, positions up to a million.
        {"name": "norm_rope packed 20011", "op": "norm_rope", "tokens": 20011, "q_heads": 28, "kv_heads": 4, "dim": 128,
         "rot": 64, "interleaved": True, "far": 1000000},
        # One token for each of 64 sequences, each into a page of its own.
        {"name": "append step 64", "op": "append", "tokens": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "scattered": True},
        # The tiny configuration's 2,048 tokens of 64 channels, odd by one.
        {"name": "append prompt 2047x64", "op": "append", "tokens": 2047, "kv_heads": 8, "dim": 64, "page": 16,
         "scattered": False},
        # A long-context prompt into permuted pages.
        {"name": "append prompt 32768", "op": "append", "tokens": 32768, "kv_heads": 4, "dim": 128, "page": 64,
         "scattered": False},
        # A single user, a short context: latency.
        {"name": "attend 1x777", "op": "attend", "batch": 1, "longest": 777, "ragged": 0, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "weights": False},
        # A serving batch whose contexts differ widely.
        {"name": "attend 64 ragged 8192", "op": "attend", "batch": 64, "longest": 8192, "ragged": 5, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "weights": False},
        # Long contexts with 7 query heads per kv head, weights added up.
        {"name": "attend 16x32768 weights", "op": "attend", "batch": 16, "longest": 32768, "ragged": 0, "q_heads": 28,
         "kv_heads": 4, "dim": 128, "page": 64, "weights": True},
        # A small cache of 64-channel heads cut to half.
        {"name": "evict 4x2048 half", "op": "evict", "batch": 4, "longest": 2048, "ragged": 0, "kv_heads": 8, "dim": 64,
         "page": 16, "keep": 1024, "recent": 128},
        # A serving batch cut to half its longest context.
        {"name": "evict 16 ragged 8192", "op": "evict", "batch": 16, "longest": 8192, "ragged": 3, "kv_heads": 8,
         "dim": 128, "page": 64, "keep": 4096, "recent": 512},
        # Long contexts that went one page over their budget.
        {"name": "evict 8x32768 a page", "op": "evict", "batch": 8, "longest": 32768, "ragged": 0, "kv_heads": 4,
         "dim": 128, "page": 64, "keep": 32704, "recent": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "evict"])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm_rope":
        return {"op": op, "tokens": _log(rng, 1, 16000), "q_heads": kv * rng.choice([1, 3, 4, 7, 8]), "kv_heads": kv,
                "dim": rng.choice([64, 128, 256]) if kv < 4 else dim, "rot": rng.choice([32, 48, 64]),
                "interleaved": rng.random() < 0.5, "far": _log(rng, 100, 1000000)}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 16000), "kv_heads": kv, "dim": dim, "page": page,
                "scattered": rng.random() < 0.4}
    batch = _log(rng, 1, 64)
    longest = _log(rng, 2, 1800000 // (batch * kv) if op == "attend" else min(65536, 900000 // (batch * kv)))
    longest = min(longest, 131072)
    ragged = rng.randrange(1, 1000) if rng.random() < 0.7 else 0
    if op == "attend":
        return {"op": op, "batch": batch, "longest": longest, "ragged": ragged,
                "q_heads": kv * rng.choice([1, 2, 4, 7, 8, 12]), "kv_heads": kv, "dim": dim, "page": page,
                "weights": rng.random() < 0.5}
    keep = max(1, int(longest * rng.uniform(0.2, 0.99)))
    return {"op": op, "batch": batch, "longest": longest, "ragged": ragged, "kv_heads": kv, "dim": dim, "page": page,
            "keep": keep, "recent": rng.randrange(0, keep + 1)}


def _lens(case):
    """Context lengths: all the longest, or log-uniform from 1 up to it (by the
    case alone), the first one the longest."""
    if not case["ragged"]:
        return [case["longest"]] * case["batch"]
    rng = random.Random(case["ragged"])
    return [case["longest"]] + [_log(rng, 1, case["longest"]) for _ in range(case["batch"] - 1)]


def _token_bytes(dim):
    return dim + dim // 8  # K and V of one token and kv head: 4-bit codes and a bf16 scale per 32 channels


def work(case):
    op, d = case["op"], case["dim"]
    if op == "norm_rope":
        values = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * d
        return {"bytes": 4 * values + 4 * case["tokens"], "flops": 10 * values}
    if op == "append":
        rows = case["tokens"] * case["kv_heads"]
        return {"bytes": rows * (4 * d + _token_bytes(d) + _token_bytes(d) + 4 * d) + 8 * case["tokens"],
                "flops": 8 * rows * d}
    lens = _lens(case)
    tokens = sum(lens) * case["kv_heads"]
    if op == "attend":
        rows = case["batch"] * case["q_heads"]
        extra = 8 * tokens + 4 * rows if case["weights"] else 0
        return {"bytes": tokens * _token_bytes(d) + 4 * rows * d + extra, "flops": 4 * sum(lens) * case["q_heads"] * d}
    # Weights and positions are read once; a token whose slot lies past the
    # kept ones moves into the slot of an evicted one: for weights that do not
    # depend on the slot that is (n - keep) * keep / n moves, without the
    # protected ones, which all lie at the end here.
    moves = 0.0
    for n in lens:
        if n > case["keep"]:
            tail = n - case["keep"]
            sure = min(case["recent"], tail)
            free = n - min(case["recent"], n)
            moves += sure + (tail - sure) * (case["keep"] - min(case["recent"], n)) / max(1, free)
    moves *= case["kv_heads"]
    return {"bytes": 8 * tokens + moves * 2 * (_token_bytes(d) + 8), "flops": tokens}


# ---- the cache format, in torch ---------------------------------------------------

def _quantise(x):
    """(codes 1..15 uint8 [..., D], scales bf16 [..., D/32]) of x [..., D]."""
    x = x.float().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    s = (top / torch.full_like(top, 7.0)).to(torch.bfloat16)
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    usable = fine & (s > 0)
    c = torch.round(x / torch.where(usable, s.float(), 1.0)[..., None]).clamp(-7, 7)
    c = torch.where(usable[..., None], c, 0.0) + 8
    return c.to(torch.uint8).flatten(-2), torch.where(fine, s, torch.nan)


def _pack_cells(k, v):
    """Cells [..., 18 * D] uint8 of K, V [..., 16, D]."""
    d = k.shape[-1]
    lead = k.shape[:-2]
    gr = d // 32
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    n = len(lead)

    def order(x, dims):
        return x.permute(*range(n), *(n + i for i in dims))

    kc = order(kc.view(*lead, 16, gr, 4, 2, 4), (0, 2, 1, 3, 4)).reshape(*lead, -1, 2)
    vc = order(vc.view(*lead, 2, 4, 2, gr, 8, 4), (0, 4, 1, 3, 2, 5)).reshape(*lead, -1, 2)
    parts = [kc[..., 0] | (kc[..., 1] << 4), vc[..., 0] | (vc[..., 1] << 4)]
    for s in (ks, vs):
        parts.append(order(s.view(*lead, 8, 2, gr), (0, 2, 1)).reshape(*lead, -1).contiguous().view(torch.uint8))
    return torch.cat(parts, -1)


def _unpack_cells(cells, d):
    """K, V [..., 16, D] fp32 of cells [..., 18 * D] uint8."""
    lead = cells.shape[:-1]
    gr = d // 32
    n = len(lead)
    kc, vc, ks, vs = cells.split((8 * d, 8 * d, d, d), -1)

    def order(x, dims):
        return x.permute(*range(n), *(n + i for i in dims))

    def codes(c):
        return torch.stack((c & 15, c >> 4), -1).float() - 8

    def scales(s):
        return order(s.contiguous().view(torch.bfloat16).view(*lead, 8, gr, 2), (0, 2, 1)).reshape(*lead, 16, gr).float()

    k = order(codes(kc).view(*lead, 16, 4, gr, 2, 4), (0, 2, 1, 3, 4)).reshape(*lead, 16, gr, 32)
    v = order(codes(vc).view(*lead, 2, 8, 4, gr, 2, 4), (0, 2, 4, 3, 1, 5)).reshape(*lead, 16, gr, 32)
    return (k * scales(ks)[..., None]).flatten(-2), (v * scales(vs)[..., None]).flatten(-2)


def _token_words(dim):
    """Word offsets inside a cell of each of its 16 tokens' 16-bit words:
    [16, 9 * D / 16], in the order K codes, V codes, K scales, V scales."""
    gr = dim // 32
    t = torch.arange(16, device=DEV)[:, None]
    pair = t // 2 * gr * 2 + t % 2
    kc = t * (dim // 4) + torch.arange(dim // 4, device=DEV)
    g, i = torch.arange(8, device=DEV)[:, None], torch.arange(gr, device=DEV)
    vc = 4 * dim + (t // 8 * 32 + t % 8 // 2) * gr * 2 + t % 2 + (g * 4 * gr * 2 + i * 2).reshape(1, -1)
    ks = 8 * dim + pair + 2 * i
    return torch.cat((kc, vc, ks, ks + dim // 2), 1)


# ---- what a program has in hand ----------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _kv_rows(g, tokens, heads, dim):
    """K with a scale of its own per head and channel and V plain: the
    structure of the synthetic KV tensors."""
    scale = torch.exp(0.6 * _normal(g, heads, dim))
    return (_normal(g, tokens, heads, dim) * scale).to(torch.bfloat16), (_normal(g, tokens, heads, dim) * 0.5).to(torch.bfloat16)


def _paged(g, case):
    """A filled pool, its block table and lengths."""
    lens = _lens(case)
    page, heads, d = case["page"], case["kv_heads"], case["dim"]
    width = -(-max(lens) // page)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    at = torch.tensor(counts, device=DEV)
    j = torch.arange(width, device=DEV)
    first = torch.cumsum(at, 0) - at
    table = ids[(first[:, None] + torch.minimum(j, at[:, None] - 1)).clamp_min(0)].contiguous()
    k, v = _kv_rows(g, pages * page, heads, d)
    cells = [x.view(pages, page // CELL, CELL, heads, d).permute(0, 3, 1, 2, 4) for x in (k, v)]
    pool = _pack_cells(*cells).reshape(pages, heads, -1)
    return {"pool": pool, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "pages": pages}


def prepare(case, seed):
    g = _generator(seed)
    op, d = case["op"], case["dim"]
    s = {"case": case}
    if op == "norm_rope":
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        # One matrix product's output: queries, keys and values of a token side by side.
        qkv = (_normal(g, t, hq + 2 * hk, d) * 2).to(torch.bfloat16)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["wq"], s["wk"] = ((1 + 0.2 * _normal(g, d)).to(torch.bfloat16) for _ in range(2))
        s["inv_freq"] = 1.0 / 10000.0 ** (torch.arange(case["rot"] // 2, device=DEV) * 2.0 / case["rot"])
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
    elif op == "append":
        t, h, page = case["tokens"], case["kv_heads"], case["page"]
        s["k"], s["v"] = _kv_rows(g, t, h, d)
        pages = (t if case["scattered"] else -(-t // page)) + 2
        ids = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(t, device=DEV)
        if case["scattered"]:
            s["slots"] = ids[:t] * page + torch.randint(0, page, (t,), generator=g, device=DEV)
        else:
            s["slots"] = ids[i // page] * page + i % page
        s["pool"] = torch.zeros(pages, h, page * _token_bytes(d), dtype=torch.uint8, device=DEV)
    else:
        s |= _paged(g, case)
        b, h = case["batch"], case["kv_heads"]
        if op == "attend":
            s["q"] = _normal(g, b, case["q_heads"], d).to(torch.bfloat16)
            s["scale"] = 1.0 / math.sqrt(d)
            if case["weights"]:
                s["weight"] = torch.rand((s["pages"], h, case["page"]), generator=g, device=DEV)
        else:
            # Accumulated weights span many powers of two; positions are the
            # order of arrival.
            s["weight0"] = torch.exp(2 * _normal(g, s["pages"], h, case["page"]))
            s["pos0"] = torch.zeros(s["pages"], h, case["page"], dtype=torch.int32, device=DEV)
            slot = torch.arange(s["table"].shape[1] * case["page"], device=DEV)
            bi, si = torch.nonzero(slot < s["lens"][:, None], as_tuple=True)
            s["pos0"][s["table"][bi, si // case["page"]].long(), :, si % case["page"]] = si.to(torch.int32)[:, None]
            s["weight"], s["pos"] = s["weight0"].clone(), s["pos0"].clone()
            s["next"] = s["lens"].clone()
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "attend": _own_attend, "evict": _own_evict}[op](s)
    return {"norm_rope": _norm_rope, "append": _append, "attend": _attend, "evict": _evict}[op](s)


def _own_norm_rope(s):
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    q = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(s["k"].shape, dtype=torch.bfloat16, device=DEV)
    S.sz_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, s["inv_freq"], s["positions"], q, k,
                      interleaved=s["case"]["interleaved"])
    return {"q": q, "k": k}


def _own_append(s):
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    page = s["case"]["page"]
    S.sz_cache_append(s["k"], s["v"], s["slots"], s["pool"], page)
    k, v = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    S.sz_cache_read(s["pool"], page, s["slots"], k, v)
    return {"k": k, "v": v}


def _own_attend(s):
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    c = s["case"]
    if "ws" not in s:
        need = S.sz_cache_attend_workspace_size(c["batch"], c["q_heads"], c["kv_heads"], c["dim"],
                                                s["table"].shape[1] * c["page"], c["weights"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=DEV) if c["weights"] else None
    S.sz_cache_attend(s["q"], s["pool"], c["kv_heads"], c["page"], s["table"], s["lens"], s["scale"], out, s["ws"],
                      lse=lse, weight=s.get("weight"))
    return {"out": out, "lse": lse, "weight": s["weight"]} if c["weights"] else {"out": out}


def _own_evict(s):
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    c = s["case"]
    _arrive(s)
    if "ws" not in s:
        need = S.sz_cache_evict_workspace_size(c["batch"], c["kv_heads"], s["table"].shape[1] * c["page"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    lens = torch.empty_like(s["lens"])
    S.sz_cache_evict(s["pool"], c["kv_heads"], c["dim"], c["page"], s["table"], s["lens"], s["next"], c["keep"],
                     c["recent"], s["weight"], s["pos"], lens, s["ws"])
    return {"pool": s["pool"], "weight": s["weight"], "pos": s["pos"], "lens": lens}


def _arrive(s):
    """The weights and positions that the steps since the last eviction left:
    without them a second pass over the same state would find nothing to move."""
    s["weight"].copy_(s["weight0"])
    s["pos"].copy_(s["pos0"])


def _norm_rope(s):
    c = s["case"]
    # Angles of far positions lose their low bits in 32 bits.
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def head(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r.chunk(2, -1)
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, rest), -1).to(torch.bfloat16)

    return {"q": head(s["q"], s["wq"]), "k": head(s["k"], s["wk"])}


def _append(s):
    c = s["case"]
    d, page = c["dim"], c["page"]
    gr = d // 32
    # The words of a token in the order of its cell; K first, then V.
    (kc, ks), (vc, vs) = _quantise(s["k"]), _quantise(s["v"])
    t, h = kc.shape[:2]
    kn = kc.view(t, h, gr, 4, 2, 4).permute(0, 1, 3, 2, 4, 5).reshape(t, h, -1, 4).int()
    vn = vc.view(t, h, gr, 8, 4).permute(0, 1, 3, 2, 4).reshape(t, h, -1, 4).int()
    nibble = torch.tensor([1, 16, 256, 4096], device=DEV, dtype=torch.int32)
    words = torch.cat(((kn * nibble).sum(-1).to(torch.int16), (vn * nibble).sum(-1).to(torch.int16),
                       ks.view(torch.int16), vs.view(torch.int16)), -1)
    at = _word_index(s["slots"], page, h, d)
    flat = s["pool"].view(torch.int16).view(-1)
    flat[at] = words
    # Read back.
    w = flat[at]
    kn, vn, ks, vs = w.split((d // 4, d // 4, gr, gr), -1)
    shift = torch.tensor([0, 4, 8, 12], device=DEV, dtype=torch.int32)

    def values(n, scale):
        return (((n.int()[..., None] >> shift) & 15) - 8).float(), scale.contiguous().view(torch.bfloat16).float()[..., None]

    kv, ksf = values(kn, ks)
    vv, vsf = values(vn, vs)
    k = kv.view(t, h, 4, gr, 2, 4).permute(0, 1, 3, 2, 4, 5).reshape(t, h, gr, 32) * ksf
    v = vv.view(t, h, 8, gr, 4).permute(0, 1, 3, 2, 4).reshape(t, h, gr, 32) * vsf
    return {"k": k.flatten(-2).to(torch.bfloat16), "v": v.flatten(-2).to(torch.bfloat16)}


def _word_index(slots, page, heads, dim):
    """Indexes of the 16-bit words of tokens at `slots`, [T, heads, 9 * D / 16]."""
    slots = slots.long()
    head = (slots // page)[:, None] * heads + torch.arange(heads, device=DEV)
    cell = head * (page // CELL) + (slots % page // CELL)[:, None]
    return cell[..., None] * (9 * dim) + _token_words(dim)[slots % CELL][:, None]


def _attend(s):
    c = s["case"]
    b, h, d, page = c["batch"], c["kv_heads"], c["dim"], c["page"]
    pages = s["table"].long()
    cells = s["pool"].view(-1, h, page // CELL, 18 * d)[pages]
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(b, h, -1, d) for x in _unpack_cells(cells, d))
    seen = torch.arange(k.shape[2], device=DEV) < s["lens"][:, None]
    q = s["q"].float().view(b, h, -1, d)
    logit = q @ k.transpose(-1, -2) * s["scale"]
    logit = torch.where(seen[:, None, None], logit, -torch.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    p = p / total
    out = (p @ v).reshape(b, -1, d).to(torch.bfloat16)
    if not c["weights"]:
        return {"out": out}
    bi, si = torch.nonzero(seen, as_tuple=True)
    s["weight"][pages[bi, si // page], :, si % page] += p.sum(2)[bi, :, si]
    return {"out": out, "lse": (top + total.log()).reshape(b, -1), "weight": s["weight"]}


def _evict(s):
    c = s["case"]
    _arrive(s)
    page, h, d = c["page"], c["kv_heads"], c["dim"]
    pages = s["table"].long()
    n = s["lens"][:, None, None]

    def slots(x):  # [pages, heads, page] -> [batch, heads, slots]
        return x[pages].permute(0, 2, 1, 3).flatten(2)

    w, pos = slots(s["weight"]), slots(s["pos"])
    slot = torch.arange(w.shape[-1], device=DEV)
    held = (slot < n).expand_as(w)
    w = torch.where(held, torch.nan_to_num(w, nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf), -torch.inf)
    safe = held & (pos >= (s["next"] - c["recent"])[:, None, None])
    # Most wanted first: protected, then by weight, then by slot, unused slots last.
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    rank = (safe.int() + held.int()).gather(-1, order)
    order = order.gather(-1, torch.argsort(rank, dim=-1, descending=True, stable=True))
    stays = torch.zeros_like(held).scatter(-1, order[..., :c["keep"]], True) & held
    hole = torch.nonzero(held & ~stays & (slot < c["keep"]))
    mover = torch.nonzero(stays & (slot >= c["keep"]))
    words = _token_words(d)

    def at(e):
        where = pages[e[:, 0], e[:, 2] // page] * h + e[:, 1]
        cell = where * (page // CELL) + e[:, 2] % page // CELL
        return where * page + e[:, 2] % page, cell[:, None] * (9 * d) + words[e[:, 2] % CELL]

    (to, to_w), (fro, fro_w) = at(hole), at(mover)
    flat = s["pool"].view(torch.int16).view(-1)
    flat[to_w] = flat[fro_w]
    for x in (s["weight"].view(-1), s["pos"].view(-1)):
        x[to] = x[fro]
    return {"pool": s["pool"], "weight": s["weight"], "pos": s["pos"],
            "lens": torch.minimum(s["lens"], torch.full_like(s["lens"], c["keep"]))}


# ---- the definition in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["dim"]
    if op == "norm_rope":
        out = {}
        theta = torch.outer(s["positions"].double(), s["inv_freq"].double())
        turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]
        half = case["rot"] // 2
        for name in "qk":
            x = s[name].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * s["w" + name].double()
            i = torch.arange(half, device=DEV)
            re, im = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[..., re], x[..., im]) * turn
            x[..., re], x[..., im] = z.real, z.imag
            out[name] = x
        return out
    if op == "append":
        out = {}
        for name in "kv":
            x = s[name].double().view(*s[name].shape[:2], d // 32, 32)
            step = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
            out[name] = torch.where(step > 0, (x / step).round().clamp(-7, 7) * step, 0.0).flatten(-2)
        return out
    if op == "evict":
        return None  # whole numbers and moved values only
    # attend: one sequence at a time, every code found by its byte address.
    page, h = case["page"], case["kv_heads"]
    raw = s["pool"].view(-1)
    tau, ch = torch.arange(CELL, device=DEV)[:, None], torch.arange(d, device=DEV)[None]
    r = ch % 32
    kword = ((tau * 4 + r // 8) * (d // 32) + ch // 32) * 2 + r // 4 % 2
    vword = (((tau // 8 * 8 + r // 4) * 4 + tau % 8 // 2) * (d // 32) + ch // 32) * 2 + tau % 2
    group = ((tau // 2) * (d // 32) + ch // 32) * 2 + tau % 2
    out, lse = [], []
    weight = s["weight"].double() if case["weights"] else None
    for b, n in enumerate(_lens(case)):
        slot = torch.arange(n, device=DEV)
        pid = s["table"][b].long()[slot // page]
        per = -(-case["q_heads"] // h)
        for head in range(h):
            cell = ((pid * h + head) * (page // CELL) + slot % page // CELL) * (18 * d)

            def values(word, codes, scales):
                byte = raw[cell[:, None] + codes + word[slot % CELL] * 2 + (ch % 4) // 2].int()
                code = torch.where(ch % 2 == 1, byte >> 4, byte & 15) - 8
                at = (cell[:, None] + scales) // 2 + group[slot % CELL]
                return code.double() * raw.view(torch.bfloat16)[at].double()

            k, v = values(kword, 0, 16 * d), values(vword, 8 * d, 17 * d)
            q = s["q"][b, head * per:(head + 1) * per].double()
            z = (q @ k.T) * s["scale"]
            total = torch.logsumexp(z, -1, keepdim=True)
            p = (z - total).exp()
            out.append(p @ v)
            lse.append(total[:, 0])
            if weight is not None:
                weight[pid, head, slot % page] += p.sum(0)
    res = {"out": torch.cat(out).view(case["batch"], -1, d)}
    if weight is not None:
        res |= {"lse": torch.cat(lse).view(case["batch"], -1), "weight": weight}
    return res
