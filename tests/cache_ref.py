"""Plain 64-bit reference of the 4-bit cache operators, on the CPU.

Written from the formulas in include/splitzip.h; shares no code with the
kernels.
"""
import math

import torch

FLT_MIN = 2.0 ** -126


def normal_bf16(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---- format ----------------------------------------------------------------------

def page_bytes(dim, heads, page):
    return heads * page * (dim + dim // 8)


def words_of_token(dim, off):
    """16-bit word numbers in a page's head run (cells of 9 dim words) of the
    token at offset off: (K words [dim/4] of channels 4w.., V words, K scale
    words [dim/32], V scale words)."""
    base, t, gr = off // 16 * 9 * dim, off % 16, dim // 32
    kw, vw = [], []
    for c in range(0, dim, 4):
        i, r = c // 32, c % 32
        q, h = r // 8, r % 8 // 4
        kw.append(base + ((t * 4 + q) * gr + i) * 2 + h)
        vw.append(base + 4 * dim + (((t // 8 * 8 + r // 4) * 4 + t % 8 // 2) * gr + i) * 2 + t % 2)
    ks = [base + 8 * dim + (t // 2 * gr + i) * 2 + t % 2 for i in range(gr)]
    vs = [w + dim // 2 for w in ks]
    return kw, vw, ks, vs


def quantise(x):
    """(codes int [..., D], scales float64 [..., D/32]) of bf16 x [..., D]."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    s = (torch.where(bad, 0.0, top) / 7).to(torch.bfloat16).double()
    s = torch.where(s < FLT_MIN, 0.0, s)
    q = torch.where((s > 0)[..., None] & ~bad[..., None], torch.nan_to_num(x) / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    codes = q.round().clamp(-7, 7).long() + 8
    return codes.flatten(-2), torch.where(bad, math.nan, s)


def dequantise(codes, scales):
    return ((codes - 8).double().unflatten(-1, (-1, 32)) * scales[..., None]).flatten(-2)


def store(pool, k, v, slots, page):
    """Writes K, V [T, H, D] into pool (uint8 [pages, bytes], CPU) at slots."""
    _, heads, dim = k.shape
    w = pool.view(torch.int16).view(pool.shape[0], heads, -1)
    (kc, ks), (vc, vs) = quantise(k), quantise(v)
    shift = torch.tensor([1, 16, 256, 4096])

    def word(c):
        x = (c.unflatten(-1, (-1, 4)) * shift).sum(-1)
        return torch.where(x >= 32768, x - 65536, x).to(torch.int16)

    kw, vw = word(kc), word(vc)
    bits = [s.to(torch.bfloat16).view(torch.int16) for s in (ks, vs)]
    for i, slot in enumerate(slots.tolist()):
        if not 0 <= slot < pool.shape[0] * page:
            continue
        at = words_of_token(dim, slot % page)
        for part, src in zip(at, (kw[i], vw[i], bits[0][i], bits[1][i])):
            w[slot // page][:, part] = src
    return pool


def load(pool, slots, page, heads, dim):
    """float64 K, V [T, H, D] at slots (pool: uint8 CPU [pages, bytes])."""
    w = pool.view(torch.int16).view(pool.shape[0], heads, -1)
    shift = torch.tensor([0, 4, 8, 12])
    ks, vs = [], []
    for slot in slots.tolist():
        kw, vw, sk, sv = words_of_token(dim, slot % page)
        row = w[slot // page]
        for out, words, sc in ((ks, kw, sk), (vs, vw, sv)):
            codes = (row[:, words].long()[..., None] >> shift & 15).flatten(-2)
            out.append(dequantise(codes, row[:, sc].contiguous().view(torch.bfloat16).double()))
    empty = torch.zeros(0, heads, dim, dtype=torch.float64)
    return (torch.stack(ks), torch.stack(vs)) if ks else (empty, empty)


def fill(gen_, pages, heads, page, dim, scale=1.0):
    """A pool whose every slot holds a quantised random token."""
    pool = torch.zeros(pages, page_bytes(dim, heads, page), dtype=torch.uint8)
    n = pages * page
    k = normal_bf16(gen_, n, heads, dim, scale=scale)
    v = normal_bf16(gen_, n, heads, dim)
    return store(pool, k, v, torch.arange(n), page)


# ---- operators ----------------------------------------------------------------------

def norm_rope(x, w, eps, inv_freq, positions, interleaved):
    """(result float64, size of what enters each value's sum) of x [T, H, D]."""
    rot = 2 * inv_freq.numel()
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y, size = x.clone(), x.abs()
    both = x[..., a].abs() + x[..., b].abs()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    size[..., a] = both
    size[..., b] = both
    return y, size


def attend(q, k, v, scale):
    """One sequence: q [Hq, D], k, v float64 [n, H, D].  Returns (out, sum of
    weight * |v|, lse, weights [H, n], largest sum of what a kernel adds up for
    a logit: |scale q| (|code - 8| + 8) s, with 7 s the largest |k| of a group)."""
    hq, d = q.shape
    n, h, _ = k.shape
    if n == 0:
        return torch.zeros(hq, d).double(), torch.zeros(hq, d).double(), torch.full((hq,), -math.inf).double(), \
            torch.zeros(h, 0).double(), 0.0
    qg = q.double().view(h, -1, d)
    s = torch.einsum("hgd,nhd->hgn", qg, k) * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    out = torch.einsum("hgn,nhd->hgd", p, v)
    mag = torch.einsum("hgn,nhd->hgd", p, v.abs())
    kk = (k.abs().unflatten(-1, (-1, 32)) + 8 / 7 * k.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)).flatten(-2)
    reach = float((torch.einsum("hgd,nhd->hgn", qg.abs(), kk) * abs(scale)).max())
    return out.reshape(hq, d), mag.reshape(hq, d), lse.reshape(hq), p.sum(1), reach


def evict_plan(weight, pos, next_pos, keep, recent):
    """One sequence and head: [(target slot, source slot)] for weights [n]."""
    n = len(weight)
    if n <= keep:
        return []
    w = [-math.inf if math.isnan(x) else x for x in weight]
    order = sorted(range(n), key=lambda i: (not pos[i] >= next_pos - recent, -w[i], i))
    stays = set(order[:keep])
    return list(zip([i for i in range(keep) if i not in stays], [i for i in range(keep, n) if i in stays]))
