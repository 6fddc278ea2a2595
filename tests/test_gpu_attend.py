"""Attention over the 4-bit cache against the formula in 64 bits on the values
that the cache holds.

Tolerances.  A logit is an fp32 sum of D products in the matrix unit (whose
additions may truncate: 2^-23 each), of the group offsets and of the scaled
groups: (D + 16) * 2^-23 of the sum of the terms' sizes.  Output: a weight
times its scale is rounded to bf16 (2^-8 of sum p |v|), sums are fp32, the
result is rounded to bf16 (2^-8 of it); a logit's error is a factor of its
weight and of the normaliser.  Log-sum and accumulated weights stay in fp32:
2^-18 of their size (approximate exponentials, sums) and the logits' error.
"""
import math

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

S = None


@pytest.fixture(autouse=True)
def _lib():
    global S
    from lossless_kv_cache_bf16_gb300 import splitzip

    S = splitzip


def make(lens, heads, group, dim, page, seed, spare=2, k_scale=1.0):
    """(pool CPU, table, lens, q): sequences in permuted pages, every slot of
    the pool, held or not, filled."""
    g = R.gen(seed)
    counts = [max(1, -(-n // page)) for n in lens]
    pages = sum(counts) + spare
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    pool = R.fill(g, pages, heads, page, dim, scale=k_scale)
    q = R.normal_bf16(g, len(lens), heads * group, dim)
    return pool, table, torch.tensor(lens, dtype=torch.int32), q


def run(pool, table, lens, q, heads, page, scale, weight=None, status=True):
    b, hq, d = q.shape
    need = S.sz_cache_attend_workspace_size(b, hq, heads, d, table.shape[1] * page, weight is not None)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q.cuda(), float("nan"))
    lse = torch.full((b, hq), float("nan"), device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda") if status else None
    S.sz_cache_attend(q.cuda(), pool.cuda(), heads, page, table.cuda(), lens.cuda(), scale, out, ws, lse=lse, weight=weight,
                      status=st)
    torch.cuda.synchronize()
    return out, lse, int(st) if status else 0


def slots_of(table_row, n, page):
    s = torch.arange(n)
    return table_row[s // page].long() * page + s % page


def check_rows(out, want, mag, reach, d):
    logit = (d + 16) * 2.0 ** -23 * reach
    tol = 2.0 ** -8 * 1.01 * (mag + want.abs()) + (2 * logit + 2.0 ** -17) * mag + 1e-30
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def check(out, lse, pool, table, lens, q, heads, page, scale, weight0=None, weight=None):
    d = q.shape[2]
    wref = None if weight is None else weight0.double().clone()
    wtol = None if weight is None else 2.0 ** -23 * weight0.double().abs()
    for b, n in enumerate(lens.tolist()):
        slots = slots_of(table[b], n, page)
        k, v = R.load(pool, slots, page, heads, d)
        want, mag, wlse, w, reach = R.attend(q[b], k, v, scale)
        check_rows(out[b], want, mag, reach, d)
        logit = (d + 16) * 2.0 ** -23 * reach
        size = 1 + (float(wlse.abs().max()) if n else 0.0)
        if lse is not None:
            got = lse[b].double().cpu()
            if n == 0:
                assert bool((got == -math.inf).all())
            else:
                assert bool(((got - wlse).abs() <= logit + 2.0 ** -18 * size).all()), (b, n)
        if weight is not None:
            wref[slots // page, :, slots % page] += w.T
            wtol[slots // page, :, slots % page] += w.T * (2 * logit + 2.0 ** -17 * size + 2.0 ** -23) + 2.0 ** -100
    if weight is not None:
        err = (weight.double().cpu() - wref).abs()
        assert bool((err <= wtol * 1.01).all()), float((err - wtol).max())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 9, 16, 20])
def test_groups(dim, group):
    heads, page = 2, 16
    pool, table, lens, q = make([1, 45, 200], heads, group, dim, page, seed=group + dim)
    scale = dim ** -0.5
    out, lse, st = run(pool, table, lens, q, heads, page, scale)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, scale)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 1024])
def test_lengths_around_cells_units_and_pages(page, weighted):
    heads, group, dim = 2, 4, 128
    sizes = [0, 1, 2, 15, 16, 17, 31, 32, 33, 0, 47, 48, 49, 63, 64, 65, 127, 128, 129, 0]
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=page)
    weight0 = torch.rand(pool.shape[0], heads, page, generator=R.gen(1))
    weight = weight0.cuda() if weighted else None
    out, lse, st = run(pool, table, lens, q, heads, page, 0.09, weight=weight)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.09, weight0, weight)


@pytest.mark.parametrize("batch,longest,heads,group,dim,page", [
    (1, 5000, 1, 8, 128, 64),      # one item over many warps and blocks
    (1, 3001, 8, 4, 64, 16),
    (2, 2500, 4, 12, 128, 128),    # 16-head items over warps and blocks
    (40, 300, 2, 7, 128, 32),
    (600, 40, 4, 2, 64, 16),       # many items per warp
])
@pytest.mark.parametrize("weighted", [False, True])
def test_splits(batch, longest, heads, group, dim, page, weighted):
    g = R.gen(batch)
    sizes = [longest] + torch.randint(0, longest + 1, (batch - 1,), generator=g).tolist()
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=batch + longest)
    weight0 = torch.zeros(pool.shape[0], heads, page)
    weight = weight0.cuda() if weighted else None
    scale = dim ** -0.5
    out, lse, st = run(pool, table, lens, q, heads, page, scale, weight=weight)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, scale, weight0, weight)
    again, lse2, _ = run(pool, table, lens, q, heads, page, scale, weight=weight0.cuda() if weighted else None)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("k_scale,q_scale,scale", [(30.0, 1.0, 0.3), (1.0, 2.0 ** 40, 2.0 ** -42), (2.0 ** -60, 2.0 ** 58, 0.2),
                                                   (1.0, 1.0, 0.0), (1.0, 1.0, -0.1), (1.0, 0.0, 0.1)])
def test_ranges(k_scale, q_scale, scale):
    """Weights that span hundreds of powers of two, large and small queries and
    keys, no and negative softmax scale, zero queries."""
    heads, group, dim, page = 2, 5, 128, 32
    pool, table, lens, q = make([700, 90, 1], heads, group, dim, page, seed=5, k_scale=k_scale)
    q = q * q_scale
    out, lse, st = run(pool, table, lens, q, heads, page, scale)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, scale)


def test_rising_logits():
    """A maximum that grows along the sequence, past the step at which the
    running maximum moves, and one that falls."""
    heads, group, dim, page = 1, 4, 128, 64
    g = R.gen(2)
    n = 900
    q = torch.ones(2, heads * group, dim).to(torch.bfloat16)
    slope = torch.linspace(0, 60, n)
    for b, s in enumerate((slope, slope.flip(0))):
        k = (s[:, None, None] / dim + 0.01 * torch.randn(n, heads, dim, generator=g)).to(torch.bfloat16)
        v = R.normal_bf16(g, n, heads, dim)
        pages = -(-n // page)
        pool = R.store(torch.zeros(pages, R.page_bytes(dim, heads, page), dtype=torch.uint8), k, v, torch.arange(n), page)
        table = torch.arange(pages, dtype=torch.int32)[None]
        lens = torch.tensor([n], dtype=torch.int32)
        out, lse, st = run(pool, table, lens, q[b:b + 1], heads, page, 1.0)
        assert st == 0
        check(out, lse, pool, table, lens, q[b:b + 1], heads, page, 1.0)


@pytest.mark.parametrize("weighted", [False, True])
def test_slots_past_the_length_may_hold_anything(weighted):
    heads, group, dim, page = 2, 4, 128, 64
    sizes = [1, 15, 16, 33, 70, 0]
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=31)
    clean, lse, _ = run(pool, table, lens, q, heads, page, 0.1)
    dirty = torch.full_like(pool, 0xFF)                       # every scale a NaN
    for b, n in enumerate(sizes):
        w, src = dirty.view(torch.int16).view(pool.shape[0], heads, -1), pool.view(torch.int16).view(pool.shape[0], heads, -1)
        for slot in slots_of(table[b], n, page).tolist():
            for part in R.words_of_token(dim, slot % page):
                w[slot // page][:, part] = src[slot // page][:, part]
    weight = torch.zeros(pool.shape[0], heads, page, device="cuda") if weighted else None
    out, lse2, st = run(dirty, table, lens, q, heads, page, 0.1, weight=weight)
    assert st == 0 and torch.equal(out, clean) and torch.equal(lse, lse2)
    if weighted:
        assert bool(torch.isfinite(weight).all())
        held = torch.zeros(pool.shape[0], page, dtype=torch.bool)
        for b, n in enumerate(sizes):
            s = slots_of(table[b], n, page)
            held[s // page, s % page] = True
        assert bool((weight.cpu().transpose(1, 2)[~held] == 0).all())


def test_nan_stays_in_its_sequence_and_head():
    heads, group, dim, page = 2, 3, 64, 16
    pool, table, lens, q = make([40, 40, 40], heads, group, dim, page, seed=8)
    clean, _, _ = run(pool, table, lens, q, heads, page, 0.1)
    slot = int(slots_of(table[1], 40, page)[20])
    w = pool.view(torch.int16).view(pool.shape[0], heads, -1)
    w[slot // page, 1, R.words_of_token(dim, slot % page)[2][0]] = 0x7FFF
    out, _, st = run(pool, table, lens, q, heads, page, 0.1)
    assert st == 0
    assert bool(torch.isnan(out[1, group:]).all())
    keep = torch.ones(3, heads * group, dtype=torch.bool)
    keep[1, group:] = False
    assert torch.equal(out[keep.cuda()], clean[keep.cuda()])


@pytest.mark.parametrize("weighted", [False, True])
def test_bad_lengths_and_pages_are_reported(weighted):
    heads, group, dim, page = 2, 4, 128, 16
    pool, table, lens, q = make([40, 40, 40, 40, 40], heads, group, dim, page, seed=9)
    weight = torch.zeros(pool.shape[0], heads, page, device="cuda") if weighted else None
    bad = lens.clone()
    bad[1], bad[3] = -7, table.shape[1] * page + 1
    out, lse, st = run(pool, table, bad, q, heads, page, 0.1, weight=weight)
    assert st == S.SZ_ERR_INVALID_ARG
    bad[1] = bad[3] = 0
    check(out, lse, pool, table, bad, q, heads, page, 0.1)
    wrong = table.clone()
    wrong[0, 1], wrong[2, 0], wrong[4, 2] = pool.shape[0], -1, 2 ** 31 - 1
    out, lse, st = run(pool, wrong, lens, q, heads, page, 0.1, weight=weight)
    assert st == S.SZ_ERR_INVALID_ARG
    if weighted:
        assert bool(torch.isfinite(weight).all())
    for b, left in ((0, [0, 2]), (2, [1, 2]), (4, [0, 1])):
        s = torch.cat([slots_of(table[b], 40, page)[16 * j:16 * j + 16] for j in left])
        k, v = R.load(pool, s, page, heads, dim)
        want, mag, _, _, reach = R.attend(q[b], k, v, 0.1)
        check_rows(out[b], want, mag, reach, dim)


def test_strided_and_unaligned_queries():
    heads, group, dim, page = 2, 4, 64, 16
    pool, table, lens, q = make([50, 3, 120], heads, group, dim, page, seed=10)
    want, _, _ = run(pool, table, lens, q, heads, page, 0.1)
    b, hq = 3, heads * group
    ws = torch.empty(S.sz_cache_attend_workspace_size(b, hq, heads, dim, table.shape[1] * page), dtype=torch.uint8, device="cuda")
    for first, width, extra in ((0, dim, 4), (1, dim, 0), (0, dim + 3, 1)):
        room = torch.zeros(first + b * (hq + extra) * width, dtype=torch.bfloat16, device="cuda")
        qs = room[first:].view(b, hq + extra, width)[:, extra:, :dim]
        qs.copy_(q)
        outs = torch.zeros_like(room)[first:].view(b, hq + extra, width)[:, extra:, :dim]
        S.sz_cache_attend(qs, pool.cuda(), heads, page, table.cuda(), lens.cuda(), 0.1, outs, ws)
        assert torch.equal(outs, want)


def test_pages_shared_by_sequences():
    heads, group, dim, page = 2, 4, 128, 16
    pool, table, lens, q = make([48, 48, 48], heads, group, dim, page, seed=12)
    table[1:] = table[0]
    weight0 = torch.zeros(pool.shape[0], heads, page)
    weight = weight0.cuda()
    out, lse, st = run(pool, table, lens, q, heads, page, 0.1, weight=weight)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.1, weight0, weight)


def test_graph_with_other_lengths_and_another_stream():
    heads, group, dim, page = 2, 4, 128, 16
    pool, table, lens, q = make([112, 16, 256], heads, group, dim, page, seed=14)
    want, _, _ = run(pool, table, lens, q, heads, page, 0.1, status=False)
    dev = [x.cuda() for x in (q, pool, table, lens)]
    ws = torch.empty(S.sz_cache_attend_workspace_size(3, 8, heads, dim, table.shape[1] * page, True), dtype=torch.uint8, device="cuda")
    out, weight = torch.empty_like(dev[0]), torch.zeros(pool.shape[0], heads, page, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    S.sz_cache_attend(dev[0], dev[1], heads, page, dev[2], dev[3], 0.1, out, ws, weight=weight, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sz_cache_attend(dev[0], dev[1], heads, page, dev[2], dev[3], 0.1, out, ws, weight=weight)
    for sizes in ([100, 7, 250], [1, 0, 33], [112, 16, 256]):
        new = torch.tensor(sizes, dtype=torch.int32)
        dev[3].copy_(new)
        weight.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out, None, pool, table, new, q, heads, page, 0.1, torch.zeros(pool.shape[0], heads, page), weight)


def test_small_workspace_and_empty_batch():
    heads, group, dim, page = 2, 4, 128, 16
    pool, table, lens, q = make([10], heads, group, dim, page, seed=15)
    need = S.sz_cache_attend_workspace_size(1, 8, heads, dim, table.shape[1] * page)
    ws = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(S.SplitZipError) as e:
        S.sz_cache_attend(q.cuda(), pool.cuda(), heads, page, table.cuda(), lens.cuda(), 0.1, torch.empty_like(q.cuda()), ws)
    assert e.value.status == S.SZ_ERR_CAPACITY
    empty = torch.empty(0, 8, dim, dtype=torch.bfloat16, device="cuda")
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    S.sz_cache_attend(empty, pool.cuda(), heads, page, torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                      torch.empty(0, dtype=torch.int32, device="cuda"), 0.1, torch.empty_like(empty), ws, status=st)
    assert int(st) == 0


def test_offsets_past_32_bits():
    heads, group, dim, page = 8, 4, 128, 64
    size = S.sz_cache_page_bytes(dim, heads, page)
    pages = 5 * 10 ** 9 // size
    small, table, lens, q = make([300], heads, group, dim, page, seed=16)
    want, _, _ = run(small, table, lens, q, heads, page, 0.1)
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    far = pages - 1 - 2 * torch.arange(table.shape[1], dtype=torch.int32)
    pool[far.long().cuda()] = small[table[0].long()].cuda()
    out, _, st = run(pool, far[None].to(torch.int32), lens, q, heads, page, 0.1)
    assert st == 0 and torch.equal(out, want)


def test_largest_batch():
    heads, group, dim, page = 1, 2, 64, 16
    sizes = [(7 * b) % 20 for b in range(2048)]
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=17)
    out, lse, st = run(pool, table, lens, q, heads, page, 0.125)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.125)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_queries_stay_in_their_head(bad):
    heads, group, dim, page = 2, 4, 128, 16
    pool, table, lens, q = make([70, 5], heads, group, dim, page, seed=18)
    clean, lse, _ = run(pool, table, lens, q, heads, page, 0.1)
    q[0, 5, 17] = bad
    out, lse2, st = run(pool, table, lens, q, heads, page, 0.1)
    assert st == 0 and not bool(torch.isfinite(out[0, 5]).any())
    keep = torch.ones(2, heads * group, dtype=torch.bool, device="cuda")
    keep[0, 5] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], lse2[keep])


def test_unaligned_weights():
    """Weights that start at an odd float are added to one by one."""
    heads, group, dim, page = 2, 3, 64, 16
    pool, table, lens, q = make([75, 16, 3], heads, group, dim, page, seed=19)
    n = pool.shape[0] * heads * page
    weight0 = torch.rand(n, generator=R.gen(2)).view(pool.shape[0], heads, page)
    room = torch.zeros(n + 2, device="cuda")
    weight = room[1:-1].view(pool.shape[0], heads, page)
    weight.copy_(weight0)
    out, lse, st = run(pool, table, lens, q, heads, page, 0.1, weight=weight)
    assert st == 0 and float(room[0]) == 0 and float(room[-1]) == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.1, weight0, weight)


@pytest.mark.parametrize("heads,group,dim", [(1, 130, 64), (3, 33, 128)])
def test_many_query_heads(heads, group, dim):
    page = 32
    pool, table, lens, q = make([90, 0, 1], heads, group, dim, page, seed=20)
    weight0 = torch.zeros(pool.shape[0], heads, page)
    weight = weight0.cuda()
    out, lse, st = run(pool, table, lens, q, heads, page, 0.1, weight=weight)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.1, weight0, weight)


def test_long_context_in_large_pages():
    """The log-sum and the total weight of a context of 70,001 equal keys have
    closed forms; values that alternate give their mean."""
    heads, group, dim, page, n = 1, 2, 64, 4096, 70001
    pages = -(-n // page)
    k = torch.full((1, heads, dim), 0.5, dtype=torch.bfloat16).expand(n, -1, -1).cuda()
    v = torch.where(torch.arange(n) % 2 == 0, 1.0, -3.0).to(torch.bfloat16)[:, None, None].expand(-1, heads, dim).cuda()
    pool = torch.zeros(pages, S.sz_cache_page_bytes(dim, heads, page), dtype=torch.uint8, device="cuda")
    S.sz_cache_append(k, v, torch.arange(n, device="cuda"), pool, page)
    table = torch.arange(pages, dtype=torch.int32)[None]
    q = torch.full((1, heads * group, dim), 0.25, dtype=torch.bfloat16)
    weight = torch.zeros(pages, heads, page, device="cuda")
    out, lse, st = run(pool, table, torch.tensor([n], dtype=torch.int32), q, heads, page, 0.125, weight=weight)
    assert st == 0
    # What the cache holds, before any rounding of a read.
    key, even, odd = (float(R.dequantise(*R.quantise(x.cpu()))[0]) for x in (k[0, 0], v[0, 0], v[1, 0]))
    assert abs(float(lse[0, 0]) - (0.25 * dim * key * 0.125 + math.log(n))) < 1e-4
    mean = (even * 35001 + odd * 35000) / n
    assert float((out.double() - mean).abs().max()) <= 2.0 ** -7 * abs(mean) + 2.0 ** -8 * 2
    assert abs(float(weight.double().sum()) - group) < 1e-4 and bool((weight.flatten()[n:] == 0).all())


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_short_contexts_in_a_wide_table(page, weighted):
    """The same lengths with room for 8,192 tokens in the table: their items
    are dealt out to warps in runs instead of one to a block."""
    heads, group, dim = 2, 4, 128
    sizes = [0, 1, 2, 15, 16, 17, 31, 32, 33, 0, 47, 48, 49, 63, 64, 65, 127, 128, 129, 0]
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=page + 1)
    narrow, lse0, _ = run(pool, table, lens, q, heads, page, 0.09)
    table = torch.cat((table, torch.full((len(sizes), 8192 // page - table.shape[1]), -1, dtype=torch.int32)), 1)
    weight0 = torch.rand(pool.shape[0], heads, page, generator=R.gen(1))
    weight = weight0.cuda() if weighted else None
    out, lse, st = run(pool, table, lens, q, heads, page, 0.09, weight=weight)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.09, weight0, weight)
    check(narrow, lse0, pool, table, lens, q, heads, page, 0.09)


@pytest.mark.parametrize("tokens", [1, 383, 384, 385, 767, 768, 1152, 1535, 1536])
@pytest.mark.parametrize("heads,group", [(1, 8), (40, 1), (8, 9), (2, 20)])
def test_items_of_their_own_blocks(tokens, heads, group):
    """Lengths around the units that a block's warps share out, up to and past
    the widest table that takes this way."""
    dim, page = 64, 128
    n, width = tokens, -(-tokens // page)
    pool, table, lens, q = make([n, max(0, n - 37)], heads, group, dim, page, seed=tokens + heads)
    table = torch.cat((table, torch.full((2, width - table.shape[1]), -1, dtype=torch.int32)), 1)
    out, lse, st = run(pool, table, lens, q, heads, page, 0.125)
    assert st == 0
    check(out, lse, pool, table, lens, q, heads, page, 0.125)


@pytest.mark.parametrize("test,args", [
    (test_groups, (64, 7)), (test_groups, (128, 20)), (test_lengths_around_cells_units_and_pages, (16, True)),
    (test_ranges, (30.0, 1.0, 0.3)), (test_ranges, (2.0 ** -60, 2.0 ** 58, 0.2)), (test_rising_logits, ()),
    (test_slots_past_the_length_may_hold_anything, (True,)), (test_nan_stays_in_its_sequence_and_head, ()),
    (test_bad_lengths_and_pages_are_reported, (True,)), (test_strided_and_unaligned_queries, ()),
    (test_pages_shared_by_sequences, ()), (test_graph_with_other_lengths_and_another_stream, ()),
    (test_non_finite_queries_stay_in_their_head, (math.inf,)), (test_unaligned_weights, ()),
    (test_many_query_heads, (3, 33, 128))])
def test_the_same_in_wide_tables(test, args, monkeypatch):
    """Small cases again with room for 16,384 tokens in the table, where items
    are dealt out to warps in runs and joined by the second kernel."""
    plain_make, plain_run = make, run

    def wide(table, page):
        return torch.cat((table, torch.full((table.shape[0], 16384 // page - table.shape[1]), -1, dtype=torch.int32)), 1)

    def wide_make(lens, heads, group, dim, page, *args, **kwargs):
        pool, table, lens, q = plain_make(lens, heads, group, dim, page, *args, **kwargs)
        return pool, wide(table, page), lens, q

    def wide_run(pool, table, lens, q, heads, page, *args, **kwargs):
        return plain_run(pool, wide(table, page), lens, q, heads, page, *args, **kwargs)

    monkeypatch.setitem(globals(), "make", wide_make)
    monkeypatch.setitem(globals(), "run", wide_run)
    test(*args)
