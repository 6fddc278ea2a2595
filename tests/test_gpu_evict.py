"""Eviction against a plain selection: which tokens stay, where they go, and
that nothing else changes.  Everything is compared exactly."""
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


def make(lens, heads, dim, page, seed, width=None):
    g = R.gen(seed)
    counts = [max(1, -(-n // page)) for n in lens]
    pages = sum(counts) + 1
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(counts)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = ids[at:at + c]
        at += c
    pool = torch.randint(0, 256, (pages, R.page_bytes(dim, heads, page)), generator=g, dtype=torch.uint8)
    weight = torch.exp(3 * torch.randn(pages, heads, page, generator=g))
    pos = torch.randint(0, 1 << 30, (pages, heads, page), generator=g, dtype=torch.int32)
    for b, n in enumerate(lens):
        s = torch.arange(n)
        pos[table[b][s // page].long(), :, s % page] = s.to(torch.int32)[:, None].expand(-1, heads)
    return pool, table, torch.tensor(lens, dtype=torch.int32), weight, pos


def reference(pool, table, lens, weight, pos, next_pos, heads, dim, page, keep, recent):
    pool, weight, pos = pool.clone(), weight.clone(), pos.clone()
    words = pool.view(torch.int16).view(pool.shape[0], heads, -1)
    for b, n in enumerate(lens.tolist()):
        if not 0 <= n <= table.shape[1] * page:
            continue
        at = [(int(table[b, s // page]), s % page) for s in range(n)]
        for h in range(heads):
            w = [float(weight[p, h, o]) for p, o in at]
            ps = [int(pos[p, h, o]) for p, o in at]
            for to, fro in R.evict_plan(w, ps, int(next_pos[b]), keep, recent):
                (p0, o0), (p1, o1) = at[to], at[fro]
                for a, c in zip(R.words_of_token(dim, o0), R.words_of_token(dim, o1)):
                    words[p0, h, a] = words[p1, h, c]
                weight[p0, h, o0], pos[p0, h, o0] = weight[p1, h, o1], pos[p1, h, o1]
    new = torch.where((lens >= 0) & (lens <= table.shape[1] * page), lens.clamp(max=keep), 0).to(torch.int32)
    return pool, weight, pos, new


def run(pool, table, lens, weight, pos, next_pos, heads, dim, page, keep, recent):
    dev = [x.cuda() for x in (pool, weight, pos)]
    need = S.sz_cache_evict_workspace_size(lens.numel(), heads, table.shape[1] * page)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    new = torch.full((lens.numel(),), -9, dtype=torch.int32, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    S.sz_cache_evict(dev[0], heads, dim, page, table.cuda(), lens.cuda(), next_pos.cuda(), keep, recent, dev[1], dev[2], new, ws, status=st)
    torch.cuda.synchronize()
    return [x.cpu() for x in dev] + [new.cpu()], int(st)


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int32) if a.is_floating_point() else a, b.view(torch.int32) if b.is_floating_point() else b)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("lens,keep,recent", [
    ([1], 1, 0), ([2], 1, 0), ([2], 1, 1), ([40, 0, 33, 100], 32, 8), ([31, 32, 33, 64, 65], 32, 0),
    ([300, 299], 50, 50), ([300], 50, 60), ([300], 299, 5), ([1500, 700], 800, 100), ([257], 7, 3)])
def test_matches_the_selection(dim, page, lens, keep, recent):
    heads = 2
    pool, table, n, weight, pos = make(lens, heads, dim, page, seed=sum(lens) + keep)
    got, st = run(pool, table, n, weight, pos, n, heads, dim, page, keep, recent)
    assert st == 0
    same(got, reference(pool, table, n, weight, pos, n, heads, dim, page, keep, recent))


@pytest.mark.parametrize("kind", ["equal", "few values", "specials", "signed", "close", "all protected", "none held late"])
def test_weights(kind):
    heads, dim, page, keep, recent = 3, 64, 16, 120, 20
    lens = [500, 130, 121]
    pool, table, n, weight, pos = make(lens, heads, dim, page, seed=3)
    g = R.gen(4)
    next_pos = n.clone()
    if kind == "equal":
        weight.fill_(0.25)
    elif kind == "few values":
        weight = torch.randint(0, 3, weight.shape, generator=g).float()
    elif kind == "specials":
        pick = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1.0, 1e-45, -1e-45, 3.4e38])
        weight = pick[torch.randint(0, len(pick), weight.shape, generator=g)]
    elif kind == "signed":
        weight = torch.randn(weight.shape, generator=g)
    elif kind == "close":
        weight = 1 + torch.randint(0, 600, weight.shape, generator=g) * 2.0 ** -23
    elif kind == "all protected":
        next_pos = torch.full_like(n, -(2 ** 31))
    elif kind == "none held late":
        next_pos = torch.full_like(n, 2 ** 31 - 1)
        pos = torch.randint(-(2 ** 31), 1000, pos.shape, generator=g, dtype=torch.int32)
    got, st = run(pool, table, n, weight, pos, next_pos, heads, dim, page, keep, recent)
    assert st == 0
    same(got, reference(pool, table, n, weight, pos, next_pos, heads, dim, page, keep, recent))


@pytest.mark.parametrize("recent", [1000, 45000])
def test_long_sequences(recent):
    heads, dim, page, keep = 1, 64, 128, 40000
    pool, table, n, weight, pos = make([60001, 200], heads, dim, page, seed=6)
    weight = (weight * 4).floor() / 4                       # ties
    got, st = run(pool, table, n, weight, pos, n, heads, dim, page, keep, recent)
    assert st == 0
    same(got, reference(pool, table, n, weight, pos, n, heads, dim, page, keep, recent))


def test_bad_lengths_are_reported_and_left_alone():
    heads, dim, page = 2, 64, 16
    pool, table, n, weight, pos = make([60, 60, 60], heads, dim, page, seed=7)
    bad = n.clone()
    bad[0], bad[2] = -1, table.shape[1] * page + 1
    got, st = run(pool, table, bad, weight, pos, n, heads, dim, page, 20, 4)
    assert st == S.SZ_ERR_INVALID_ARG
    same(got, reference(pool, table, bad, weight, pos, n, heads, dim, page, 20, 4))


def test_bad_pages_are_reported_and_not_touched():
    heads, dim, page = 2, 64, 16
    pool, table, n, weight, pos = make([64, 64], heads, dim, page, seed=8)
    wrong = table.clone()
    wrong[0, 2] = pool.shape[0]
    got, st = run(pool, wrong, n, weight, pos, n, heads, dim, page, 20, 4)
    assert st == S.SZ_ERR_INVALID_ARG
    want = reference(pool, table, n, weight, pos, n, heads, dim, page, 20, 4)
    own = table[1].long()
    for a, b in zip(got[:3], want[:3]):                     # the other sequence is cut as ever
        assert torch.equal(a[own], b[own])
    other = [p for p in range(pool.shape[0]) if p not in table.flatten().tolist()] + [int(table[0, 2])]
    for a, b in zip(got[:3], (pool, weight, pos)):
        assert torch.equal(a[other], b[other])


def test_survivors_are_all_there():
    """After the moves the first `keep` slots of each head hold exactly the
    wanted tokens, values, weights and positions together."""
    heads, dim, page, keep, n = 2, 128, 16, 70, 150
    g = R.gen(11)
    pages = -(-n // page)
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    pool = R.fill(g, pages, heads, page, dim)
    weight, pos = torch.rand(pages, heads, page, generator=g), torch.zeros(pages, heads, page, dtype=torch.int32)
    s = torch.arange(n)
    at = table[0][s // page].long()
    pos[at, :, s % page] = s.to(torch.int32)[:, None].expand(-1, heads)
    lens = torch.tensor([n], dtype=torch.int32)
    got, st = run(pool, table, lens, weight, pos, lens, heads, dim, page, keep, 10)
    assert st == 0 and int(got[3]) == keep
    slots = at * page + s % page
    k, v = R.load(pool, slots, page, heads, dim)
    k2, v2 = R.load(got[0], slots[:keep], page, heads, dim)
    for h in range(heads):
        w = weight[at, h, s % page]
        order = sorted(range(n), key=lambda i: (i < n - 10, -float(w[i]), i))[:keep]
        p = got[2][at[:keep], h, s[:keep] % page].long()
        assert sorted(p.tolist()) == sorted(order)
        assert torch.equal(k2[:, h], k[p, h]) and torch.equal(v2[:, h], v[p, h])
        assert torch.equal(got[1][at[:keep], h, s[:keep] % page], w[p])


def test_graph_replay():
    heads, dim, page = 2, 64, 16
    pool, table, n, weight, pos = make([90, 40], heads, dim, page, seed=12)
    dev = [x.cuda() for x in (pool, weight, pos, table, n)]
    ws = torch.empty(S.sz_cache_evict_workspace_size(2, heads, table.shape[1] * page), dtype=torch.uint8, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sz_cache_evict(dev[0], heads, dim, page, dev[3], dev[4], dev[4], 32, 4, dev[1], dev[2], new, ws)
    for _ in range(2):
        for d, s in zip(dev, (pool, weight, pos)):
            d.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        same([x.cpu() for x in dev[:3]] + [new.cpu()], reference(pool, table, n, weight, pos, n, heads, dim, page, 32, 4))


@pytest.mark.parametrize("batch,heads", [(128, 1), (43, 3), (70, 7), (400, 1)])
@pytest.mark.parametrize("spread", ["all", "few", "one", "none"])
def test_many_lists(batch, heads, spread):
    """More (sequence, head) pairs than threads that count their moves; moves
    in all of them, in runs with gaps, only in the last sequence, nowhere."""
    dim, page, keep, recent = 64, 16, 24, 5
    g = R.gen(batch + heads)
    n = torch.randint(0, 25, (batch,), generator=g)
    if spread == "all":
        n += 25
    elif spread == "few":
        n[::37] = 70
    elif spread == "one":
        n[-1] = 900
    lens = n.tolist()
    pool, table, lens, weight, pos = make(lens, heads, dim, page, seed=batch)
    next_pos = lens.clone()
    got, st = run(pool, table, lens, weight, pos, next_pos, heads, dim, page, keep, recent)
    assert st == 0
    same(got, reference(pool, table, lens, weight, pos, next_pos, heads, dim, page, keep, recent))


@pytest.mark.parametrize("n", [8192, 8193, 100000, 131073])
@pytest.mark.parametrize("width", [8192, 16384, 131072, 262144, 1 << 20])
def test_room_in_the_table(n, width):
    """The table's width alone chooses how many keys a thread holds and how
    many blocks share a list: few tokens in a wide table and a full one."""
    heads, dim, page = 1, 64, 128
    if n > width:
        n = width
    pool, table, lens, weight, pos = make([n, 3, n // 2], heads, dim, page, seed=n, width=width // page)
    weight = (weight * 64).floor() / 64
    keep, recent = n - 700, 300
    got, st = run(pool, table, lens, weight, pos, lens, heads, dim, page, keep, recent)
    assert st == 0
    same(got, reference(pool, table, lens, weight, pos, lens, heads, dim, page, keep, recent))
