"""A DecodeCache against a replay that never reads the cache's own values.

The replay knows each token by its position: prompt rows as they were encoded,
new values as the projection gave them, new keys from the formula.  After every
step the cache must hold exactly the quantised rows of the positions that its
own table of positions names, in the slots that the replay puts them; the
attention, the accumulated weights and the survivors of an eviction follow from
the replay's rows.

Tolerances: rotated queries and keys are rounded to bf16 once (2^-8 of the
value, 2^-18 of the sum's terms, as in tests/test_gpu_norm_rope.py); attention
and weights are those of tests/test_gpu_attend.py, the weights' errors added up
over the steps with one fp32 rounding (2^-24 of the sum) each.
"""
import math

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Replay:
    """Positions, rows and weights of every sequence and kv head."""

    def __init__(self, batch, heads, dim, room):
        self.k = torch.full((batch, room, heads, dim), math.nan).double()   # by position, as the cache holds them
        self.v = self.k.clone()
        self.weight = torch.zeros(batch, heads, room).double()              # by position
        self.slack = torch.zeros(batch, heads, room).double()
        self.held = [[[] for _ in range(heads)] for _ in range(batch)]      # positions in the order of their slots
        self.next = [0] * batch

    def append(self, b, k, v):
        """k, v: bf16 rows [tokens, heads, dim]."""
        n = k.shape[0]
        at = slice(self.next[b], self.next[b] + n)
        self.k[b, at], self.v[b, at] = R.dequantise(*R.quantise(k)), R.dequantise(*R.quantise(v))
        for held in self.held[b]:
            held.extend(range(at.start, at.stop))
        self.next[b] += n

    def rows(self, b):
        """K and V of the held tokens [n, heads, dim], head by head."""
        pick = lambda x: torch.stack([x[b, torch.tensor(p), h] for h, p in enumerate(self.held[b])], 1)
        return pick(self.k), pick(self.v)

    def evict(self, b, h, weight, keep, recent):
        """weight: the accumulated weights by slot."""
        held = self.held[b][h]
        for to, fro in R.evict_plan(weight, held, self.next[b], keep, recent):
            held[to] = held[fro]
        del held[keep:]


def encoded(S, x):
    n = x.numel()
    hist = torch.empty(S.sz_histogram_bins(S.SZ_BF16), dtype=torch.int64, device="cuda")
    cb = S.sz_calibrate(S.SZ_BF16, x, hist)
    out = torch.empty(S.sz_encoded_size(S.SZ_BF16, n, n), dtype=torch.uint8, device="cuda")
    ws = torch.empty(S.sz_workspace_size(S.SZ_BF16, n), dtype=torch.uint8, device="cuda")
    size = torch.zeros(1, dtype=torch.int64, device="cuda")
    S.sz_encode(S.SZ_BF16, cb, x, out, size, None, ws)
    return out, int(size.item())


def by_slot(x, cache, b):
    """A table of the cache [pages, heads, page] as [heads, slots] of sequence b."""
    s = torch.arange(cache.held[b])
    return x.cpu()[cache.table[b].cpu().long()[s // cache.page], :, s % cache.page].T


@pytest.mark.parametrize("budget,recent", [(None, 0), (64, 16), (48, 0), (48, 48)])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 2, 128, 16), (9, 3, 64, 32)])
def test_replay(hq, hk, d, page, budget, recent):
    from lossless_kv_cache_bf16_gb300 import decode, splitzip as S

    batch, steps = 2, 70
    g = R.gen(hq + (budget or 0) + recent)
    cache = decode.DecodeCache(batch, hq, hk, d, 200, page_tokens=page, budget=budget, recent=recent)
    replay = Replay(batch, hk, d, 200)
    for b, tokens in enumerate((90, 61)):
        # K and V differ in size, so that one cannot pass for the other.
        kv = torch.stack((R.normal_bf16(g, tokens, hk, d, scale=3), R.normal_bf16(g, tokens, hk, d, scale=0.5)))
        if b == 0:
            cache.extend_from_stream(b, *encoded(S, kv.cuda()), tokens)
        else:
            cache.extend(b, kv[0, :40].cuda(), kv[1, :40].cuda())
            cache.extend(b, kv[0, 40:].cuda(), kv[1, 40:].cuda())
        replay.append(b, kv[0], kv[1])

    evictions = []
    plain_evict = cache.evict

    def evict():
        weights = [by_slot(cache.weight, cache, b) for b in range(batch)]
        plain_evict()
        for b in range(batch):
            for h in range(hk):
                replay.evict(b, h, weights[b][h].tolist(), budget, recent)
        evictions.append(list(cache.held))

    cache.evict = evict
    freq = (10000.0 ** (-torch.arange(d // 2) * 2.0 / d)).float()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2))
    scale = 1 / math.sqrt(d)
    for _ in range(steps):
        qkv = R.normal_bf16(g, batch, hq + 2 * hk, d)
        dev = qkv.cuda()
        positions = torch.tensor(replay.next)
        before = [[list(p) for p in held] for held in replay.held]
        # The step evicts at its end: the replay's rows join first.
        rotated = []

        def join():
            got = dev.cpu()
            for lo, hi, w in ((0, hq, wq), (hq, hq + hk, wk)):
                want, size = R.norm_rope(qkv[:, lo:hi], w, EPS, freq, positions, False)
                off = (got[:, lo:hi].double() - want).abs()
                assert bool((off <= 2.0 ** -8 * 1.01 * want.abs() + 2.0 ** -18 * size).all())
            assert torch.equal(got[:, hq + hk:], qkv[:, hq + hk:])
            for b in range(batch):
                replay.append(b, got[b:b + 1, hq:hq + hk], qkv[b:b + 1, hq + hk:])
            rotated.append(got[:, :hq])

        cache.evict = lambda: (join(), attended(), evict())
        results = {}

        def attended():
            for b in range(batch):
                k, v = replay.rows(b)
                results[b] = R.attend(rotated[0][b], k, v, scale)
                weights = results[b][3]
                logit = (d + 16) * 2.0 ** -23 * results[b][4]
                size = 1 + float(results[b][2].abs().max())
                for h in range(hk):
                    at = torch.tensor(replay.held[b][h])
                    replay.weight[b, h, at] += weights[h]
                    replay.slack[b, h, at] += weights[h] * (2 * logit + 2.0 ** -17 * size + 2.0 ** -23) + 2.0 ** -24 * replay.weight[b, h, at]

        out = cache.step(dev, wq.cuda(), wk.cuda(), freq.cuda())
        cache.check()
        if not rotated:
            join()
            attended()
        pool = cache.pool.cpu()
        for b in range(batch):
            want, mag, _, _, reach = results[b]
            logit = (d + 16) * 2.0 ** -23 * reach
            tol = 2.0 ** -8 * 1.01 * (mag + want.abs()) + (2 * logit + 2.0 ** -17) * mag + 1e-30
            assert bool(((out[b].double().cpu() - want).abs() <= tol).all())
            # Every slot holds the token that the replay puts there.
            assert cache.held[b] == len(replay.held[b][0]) and int(cache.lens[b]) == cache.held[b]
            assert int(cache.next_pos[b]) == replay.next[b]
            assert by_slot(cache.pos, cache, b).tolist() == replay.held[b]
            s = torch.arange(cache.held[b])
            k, v = R.load(pool, cache.table[b].cpu().long()[s // page] * page + s % page, page, hk, d)
            want_k, want_v = replay.rows(b)
            assert torch.equal(k, want_k) and torch.equal(v, want_v)
            weight = by_slot(cache.weight, cache, b).double()
            for h in range(hk):
                at = torch.tensor(replay.held[b][h])
                assert bool(((weight[h] - replay.weight[b, h, at]).abs() <= 1.01 * replay.slack[b, h, at]).all())
        if budget is None:
            assert replay.held == [[p + [int(positions[b])] for p in held] for b, held in enumerate(before)]
    if budget is None:
        assert evictions == []
    else:
        assert len(evictions) >= 2 and all(max(held) == budget for held in evictions)
