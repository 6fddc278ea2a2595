"""The decode path as a whole: a prompt arrives as a SplitZip stream, steps
norm, rotate, append and attend, and a budget evicts.  A 64-bit replay of the
same steps from the formulas gives the attention's result and, with the
library's own accumulated weights, the tokens that stay."""
import math

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget", [None, 64])
def test_prompt_from_a_stream_and_steps(budget):
    from lossless_kv_cache_bf16_gb300 import decode, splitzip as S, workloads as W

    hq, hk, d, page, tokens, steps = 8, 2, 128, 16, 100, 40
    g = R.gen(3)
    prompts = [R.normal_bf16(g, 2, tokens - 30 * b, hk, d) for b in range(2)]
    cache = decode.DecodeCache(2, hq, hk, d, 160, page_tokens=page, budget=budget, recent=16)
    for b, kv in enumerate(prompts):
        x = kv.cuda()
        n = x.numel()
        hist = torch.empty(S.sz_histogram_bins(S.SZ_BF16), dtype=torch.int64, device="cuda")
        cb = S.sz_calibrate(S.SZ_BF16, x, hist)
        out = torch.empty(S.sz_encoded_size(S.SZ_BF16, n, n), dtype=torch.uint8, device="cuda")
        ws = torch.empty(S.sz_workspace_size(S.SZ_BF16, n), dtype=torch.uint8, device="cuda")
        size = torch.zeros(1, dtype=torch.int64, device="cuda")
        S.sz_encode(S.SZ_BF16, cb, x, out, size, None, ws)
        cache.extend_from_stream(b, out, int(size.item()), kv.shape[1])
    assert cache.held == [100, 70]
    freq = (10000.0 ** (-torch.arange(d // 2) * 2.0 / d)).float()
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2))
    evictions = 0
    for _ in range(steps):
        qkv = R.normal_bf16(g, 2, hq + 2 * hk, d)
        dev = qkv.cuda()
        before = list(cache.held)
        next_pos = cache.next_pos.cpu()
        out = cache.step(dev, wq.cuda(), wk.cuda(), freq.cuda())
        cache.check()
        q, size = R.norm_rope(qkv[:, :hq], wq, 1e-6, freq, next_pos, False)
        got = dev[:, :hq].cpu()
        assert bool(((got.double() - q).abs() <= 2.0 ** -8 * 1.01 * q.abs() + 2.0 ** -18 * size).all())
        if max(before) + 1 >= (budget or 10 ** 9) + page:
            evictions += 1
            assert cache.held == [min(n + 1, budget) for n in before]
            continue                                         # the pool is cut already
        assert cache.held == [n + 1 for n in before]
        pool = cache.pool.cpu()
        for b in range(2):
            s = torch.arange(cache.held[b])
            slots = cache.table[b].cpu().long()[s // page] * page + s % page
            k, v = R.load(pool, slots, page, hk, d)
            want, mag, _, _, reach = R.attend(got[b], k, v, 1 / math.sqrt(d))
            tol = 2.0 ** -8 * 1.01 * (mag + want.abs()) + (2 * (d + 16) * 2.0 ** -23 * reach + 2.0 ** -17) * mag
            assert bool(((out[b].double().cpu() - want).abs() <= tol).all())
            # Every held token is there once, with its own position.
            p = cache.pos.cpu()[slots // page, :, slots % page].T
            for h in range(hk):
                assert len(set(p[h].tolist())) == cache.held[b] and int(p[h].max()) == int(next_pos[b])
    assert evictions == (0 if budget is None else 3)
    assert cache.lens.tolist() == cache.held


def test_weights_add_up():
    """Each step adds one unit of weight per query head."""
    from lossless_kv_cache_bf16_gb300 import decode

    hq, hk, d = 6, 2, 64
    cache = decode.DecodeCache(1, hq, hk, d, 64, page_tokens=16)
    g = R.gen(5)
    k, v = R.normal_bf16(g, 20, hk, d).cuda(), R.normal_bf16(g, 20, hk, d).cuda()
    cache.extend(0, k, v)
    freq = torch.ones(d // 2, device="cuda")
    for i in range(5):
        cache.step(R.normal_bf16(g, 1, hq + 2 * hk, d).cuda(), None, None, freq)
        assert torch.allclose(cache.weight.sum((0, 2)), torch.full((hk,), (i + 1) * hq / hk, device="cuda"), rtol=1e-4)
    with pytest.raises(ValueError):
        cache.extend(0, k.repeat(3, 1, 1), v.repeat(3, 1, 1))


def test_the_demo_runs(capsys):
    from lossless_kv_cache_bf16_gb300 import decode

    decode._demo(tokens=512, steps=96, budget=256)
    text = capsys.readouterr().out
    assert "step 96: 608 tokens against" in text
