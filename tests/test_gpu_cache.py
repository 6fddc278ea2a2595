"""Append to and read from the 4-bit cache: the bytes are those of the
definition in 64 bits (every quotient of two bf16 values is k + 1/2 or far
from it, so the codes have one right value), nothing else is touched."""
import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

S = None
CANARY = 0x5A


@pytest.fixture(autouse=True)
def _lib():
    global S
    from lossless_kv_cache_bf16_gb300 import splitzip

    S = splitzip


def fresh_pool(pages, heads, page, dim):
    return torch.full((pages, S.sz_cache_page_bytes(dim, heads, page)), CANARY, dtype=torch.uint8)


def same_values(got, ref):
    got, ref = got.cpu(), ref.to(torch.bfloat16)
    bad = torch.isnan(ref)
    return torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], ref[~bad])


def rows(seed, tokens, heads, dim):
    """Values over many powers of two; groups that are constant, zero, tiny,
    huge and not finite among them."""
    g = R.gen(seed)
    x = torch.randn(tokens, heads, dim, generator=g) * torch.exp2(torch.randint(-20, 20, (tokens, heads, dim // 32, 1), generator=g).float()
                                                                  .expand(-1, -1, -1, 32).flatten(-2))
    x = x.to(torch.bfloat16)
    if tokens > 4:
        x[1, :, :32] = 0
        x[2, :, :32] = -1.5
        x[3, :, :32] = torch.linspace(-2.0 ** -127, 2.0 ** -126, 32).to(torch.bfloat16)
        x[4, :, :32] = torch.linspace(-3e38, 3.3e38, 32).to(torch.bfloat16)
        x[4, :, 32:64] = torch.linspace(-1e38, 1.6e38, 32).to(torch.bfloat16)
        x[0, :, 32:64] = (torch.arange(32) - 16).to(torch.bfloat16) / 2   # ties
    return x


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (5, 8, 16), (64, 4, 64), (100, 3, 32), (257, 2, 128),
                                               (33, 1, 4096)])
@pytest.mark.parametrize("order", ["run", "shifted run", "scattered"])
def test_append_then_read(dim, tokens, heads, page, order):
    pages = -(-(tokens + 7) // page) + 2
    k, v = rows(tokens, tokens, heads, dim), rows(tokens + 1, tokens, heads, dim)
    g = R.gen(3)
    if order == "scattered":
        slots = torch.randperm(pages * page, generator=g)[:tokens]
    else:
        ids = torch.randperm(pages, generator=g)
        at = torch.arange(tokens) + (7 if order == "shifted run" else 0)
        slots = ids[at // page] * page + at % page
    want = R.store(fresh_pool(pages, heads, page, dim), k, v, slots, page)
    pool = fresh_pool(pages, heads, page, dim).cuda()
    weight = torch.full((pages, heads, page), 7.0, device="cuda")
    pos = torch.full((pages, heads, page), -5, dtype=torch.int32, device="cuda")
    positions = torch.randint(0, 1 << 30, (tokens,), generator=g, dtype=torch.int32)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    S.sz_cache_append(k.cuda(), v.cuda(), slots.cuda(), pool, page, positions=positions.cuda(), weight=weight, pos=pos, status=st)
    assert int(st) == 0
    assert torch.equal(pool.cpu(), want)
    wref, pref = torch.full((pages, heads, page), 7.0), torch.full((pages, heads, page), -5, dtype=torch.int32)
    wref[slots // page, :, slots % page] = 0
    pref[slots // page, :, slots % page] = positions[:, None].expand(-1, heads)
    assert torch.equal(weight.cpu(), wref) and torch.equal(pos.cpu(), pref)
    ko, vo = torch.empty_like(k.cuda()), torch.empty_like(v.cuda())
    S.sz_cache_read(pool, page, slots.cuda(), ko, vo, status=st)
    assert int(st) == 0
    for got, ref in zip((ko, vo), R.load(want, slots, page, heads, dim)):
        assert same_values(got, ref)


def test_non_finite_groups_read_as_nan():
    k, v = rows(1, 4, 2, 64), rows(2, 4, 2, 64)
    k[0, 0, 3], k[1, 1, 40], v[3, 0, 63] = float("nan"), float("inf"), -float("inf")
    pool = fresh_pool(1, 2, 16, 64).cuda()
    slots = torch.arange(4)
    S.sz_cache_append(k.cuda(), v.cuda(), slots.cuda(), pool, 16)
    ko, vo = torch.empty_like(k.cuda()), torch.empty_like(v.cuda())
    S.sz_cache_read(pool, 16, slots.cuda(), ko, vo)
    for got, src in ((ko, k), (vo, v)):
        bad = ~torch.isfinite(src).unflatten(-1, (-1, 32)).all(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
        assert torch.equal(torch.isnan(got.cpu()), bad)
        codes, s = R.quantise(src)
        assert torch.equal(got.cpu()[~bad], R.dequantise(codes, s).to(torch.bfloat16)[~bad])


@pytest.mark.parametrize("dim", [64, 128])
def test_bad_slots_are_left_out_and_reported(dim):
    heads, page, pages = 2, 16, 3
    k, v = rows(5, 40, heads, dim), rows(6, 40, heads, dim)
    slots = torch.arange(40)
    slots[3], slots[20], slots[21], slots[39] = -1, pages * page, -2, 1 << 40
    pool, st = fresh_pool(pages, heads, page, dim).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    S.sz_cache_append(k.cuda(), v.cuda(), slots.cuda(), pool, page, status=st)
    assert int(st) == S.SZ_ERR_INVALID_ARG
    assert torch.equal(pool.cpu(), R.store(fresh_pool(pages, heads, page, dim), k, v, slots, page))
    ko, vo = torch.ones_like(k.cuda()), torch.ones_like(v.cuda())
    S.sz_cache_read(pool, page, slots.cuda(), ko, vo, status=st)
    assert int(st) == S.SZ_ERR_INVALID_ARG
    left = (slots < 0) | (slots >= pages * page)
    assert bool((ko.cpu()[left] == 0).all()) and bool((vo.cpu()[left] == 0).all())
    slots[20], slots[21], slots[39] = 20, 21, -1
    S.sz_cache_append(k.cuda(), v.cuda(), slots.cuda(), pool, page, status=st)
    assert int(st) == 0


@pytest.mark.parametrize("layout", ["packed", "transposed", "odd offset", "odd head stride"])
def test_strides_and_alignment(layout):
    tokens, heads, dim, page = 37, 3, 64, 16
    k, v = rows(7, tokens, heads, dim), rows(8, tokens, heads, dim)
    first = 1 if layout == "odd offset" else 0
    width = dim + (3 if layout == "odd head stride" else 0)

    def lay(x):
        if layout == "transposed":
            return x.cuda().transpose(0, 1).contiguous().transpose(0, 1)
        room = torch.zeros(first + tokens * 2 * heads * width, dtype=x.dtype, device="cuda")
        at = room[first:].view(tokens, 2 * heads, width)[:, heads:, :dim]
        at.copy_(x)
        return at

    slots = torch.arange(tokens)
    want = R.store(fresh_pool(3, heads, page, dim), k, v, slots, page)
    pool = fresh_pool(3, heads, page, dim).cuda()
    kd, vd = lay(k), lay(v)
    S.sz_cache_append(kd, vd, slots.cuda(), pool, page)
    assert torch.equal(pool.cpu(), want)
    S.sz_cache_read(pool, page, slots.cuda(), kd, vd)
    for got, ref in zip((kd, vd), R.load(want, slots, page, heads, dim)):
        assert same_values(got, ref)


def test_offsets_past_32_bits():
    """A pool of 5 GB: slots whose byte offsets need more than 32 bits."""
    heads, page, dim = 8, 64, 128
    size = S.sz_cache_page_bytes(dim, heads, page)
    pages = 5 * 10 ** 9 // size
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    k, v = rows(11, 32, heads, dim), rows(12, 32, heads, dim)
    slots = pages * page - 1 - 3 * torch.arange(32)
    S.sz_cache_append(k.cuda(), v.cuda(), slots.cuda(), pool, page)
    last = pool[-3:].cpu()
    want = R.store(torch.zeros_like(last), k, v, slots - (pages - 3) * page, page)
    assert torch.equal(last, want)
    assert int(pool[:-3].count_nonzero()) == 0


def test_another_stream_and_a_graph():
    heads, page, dim = 4, 16, 128
    k, v = rows(13, 20, heads, dim), rows(14, 20, heads, dim)
    slots = torch.arange(20)
    want = R.store(fresh_pool(2, heads, page, dim), k, v, slots, page)
    kd, vd, sd = k.cuda(), v.cuda(), slots.cuda()
    side = torch.cuda.Stream()
    pool = fresh_pool(2, heads, page, dim).cuda()
    side.wait_stream(torch.cuda.current_stream())
    S.sz_cache_append(kd, vd, sd, pool, page, stream=side)
    side.synchronize()
    assert torch.equal(pool.cpu(), want)
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.sz_cache_append(kd, vd, sd, pool, page)
        S.sz_cache_read(pool, page, sd, ko, vo)
    for _ in range(2):
        pool.fill_(CANARY)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.cpu(), want)
    assert same_values(ko, R.load(want, slots, page, heads, dim)[0])
