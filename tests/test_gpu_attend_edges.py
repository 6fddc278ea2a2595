"""Attention over the 4-bit cache: rows that no token reaches, waits that give
up.

Tolerances are those of tests/test_gpu_attend.py.
"""
import math

import pytest
import torch

from tests import cache_ref as R
from tests.test_gpu_attend import _lib, check, make, run  # noqa: F401  (_lib loads the library)

pytestmark = pytest.mark.gpu


def widen(table, page, room):
    """The table with room for that many tokens (None: as it is).  Wide tables
    deal items out in runs and join pieces in a second kernel."""
    if room is None:
        return table
    return torch.cat((table, torch.full((table.shape[0], room // page - table.shape[1]), -1, dtype=torch.int32)), 1)


@pytest.mark.parametrize("room", [None, 16384])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("heads,group,longest", [(2, 4, 700), (1, 12, 700), (1, 8, 5000)])
def test_sequences_of_bad_pages_alone_are_empty(heads, group, longest, weighted, room):
    """Tokens of pages outside the pool are left out; where no other is held,
    the row is that of an empty sequence: zeros, log-sum -infinity."""
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    dim, page = 128, 16
    sizes = [40, 33, longest, 5, 0]
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=40 + group)
    table[1, :] = pool.shape[0]
    table[2, ::2], table[2, 1::2] = -1, 2 ** 31 - 1
    weight0 = torch.rand(pool.shape[0], heads, page, generator=R.gen(1))
    weight = weight0.cuda() if weighted else None
    out, lse, st = run(pool, widen(table, page, room), lens, q, heads, page, 0.1, weight=weight)
    assert st == S.SZ_ERR_INVALID_ARG
    for b in (1, 2, 4):
        assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all()), b
    lens[1] = lens[2] = 0
    check(out, lse, pool, table, lens, q, heads, page, 0.1, weight0, weight)


@pytest.mark.parametrize("room", [None, 16384])
@pytest.mark.parametrize("n", [5, 32, 700])
def test_logits_past_the_range_are_no_empty_row(n, room):
    """Tokens whose logits all overflow to -infinity leave no finite row."""
    heads, group, dim, page = 1, 2, 64, 16
    pages = -(-n // page)
    k = torch.full((n, heads, dim), 2.0 ** 60).to(torch.bfloat16)
    v = R.normal_bf16(R.gen(1), n, heads, dim)
    pool = R.store(torch.zeros(pages, R.page_bytes(dim, heads, page), dtype=torch.uint8), k, v, torch.arange(n), page)
    q = torch.full((1, heads * group, dim), -2.0 ** 90).to(torch.bfloat16)
    table = widen(torch.arange(pages, dtype=torch.int32)[None], page, room)
    out, lse, st = run(pool, table, torch.tensor([n], dtype=torch.int32), q, heads, page, 1.0)
    assert st == 0 and not bool(torch.isfinite(out).any())


@pytest.mark.parametrize("room", [None, 16384])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dim,heads,group,sizes", [
    (128, 2, 4, [300, 40, 33, 0, 500]), (64, 1, 12, [700, 1]), (128, 1, 8, [6000]), (64, 4, 2, [30] * 200)])
def test_a_wait_that_gives_up_leaves_the_weights_alone(dim, heads, group, sizes, weighted, room):
    """The first block's waits give up: its rows are NaN, the others right, the
    status says so, and the accumulated weights can be used for another try."""
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    page = 16
    pool, table, lens, q = make(sizes, heads, group, dim, page, seed=50 + group)
    table = widen(table, page, room)
    b, hq = len(sizes), heads * group
    weight0 = torch.rand(pool.shape[0], heads, page, generator=R.gen(1))
    want, want_lse, st = run(pool, table, lens, q, heads, page, 0.1, weight=weight0.cuda() if weighted else None)
    assert st == 0
    need = S.sz_cache_attend_workspace_size(b, hq, heads, dim, table.shape[1] * page, weighted)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, hq, device="cuda")
    weight = weight0.cuda() if weighted else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), pool.cuda(), heads, page, table.cuda(), lens.cuda(), 0.1, out, ws)
    for _ in range(2):
        S.sz_debug_attend_stalled(*args, lse=lse, weight=weight, status=status)
        assert int(status) == S.SZ_ERR_TIMEOUT
        lost = torch.isnan(lse)
        assert bool(lost[0, 0]) and (len(sizes) == 1 or not bool(lost.all()))
        assert bool(torch.isnan(out[lost]).all())
        assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
        if weighted:
            assert torch.equal(weight.cpu(), weight0)
    S.sz_cache_attend(*args, lse=lse, weight=weight, status=status)
    assert int(status) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    check(out, lse, pool, table, lens, q, heads, page, 0.1, weight0, weight)


def test_more_list_entries_than_32_bits():
    """65 sequences of 2^26 units each, all of one page, whose lengths one warp
    adds up: 2^32 entries and more.  The short sequence behind them is the last
    of the list."""
    from lossless_kv_cache_bf16_gb300 import splitzip as S

    heads, group, dim, page, width = 1, 1, 64, 4096, 2 ** 19 - 1
    longest = width * page
    # A thread takes every 384th sequence, a warp 32 threads.
    full = list(range(32)) + list(range(384, 416)) + [768]
    batch, last = 770, 769
    assert len(full) * (longest // 32) >= 2 ** 32
    pool = R.fill(R.gen(60), 2, heads, page, dim)
    table = torch.zeros((batch, width), dtype=torch.int32, device="cuda")
    table[last] = 1
    lens = torch.zeros(batch, dtype=torch.int32)
    lens[full] = longest
    lens[last] = 77
    q = R.normal_bf16(R.gen(61), batch, heads * group, dim)
    ws = torch.empty(S.sz_cache_attend_workspace_size(batch, group, heads, dim, longest), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q.cuda(), math.nan)
    lse = torch.full((batch, group), math.nan, device="cuda")
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    S.sz_cache_attend(q.cuda(), pool.cuda(), heads, page, table, lens.cuda(), 0.1, out, ws, lse=lse, status=st)
    assert int(st) == 0
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[full]).all())
    empty = lens == 0
    assert bool((out[empty.cuda()] == 0).all()) and bool((lse[empty.cuda()] == -math.inf).all())
    check(out[last:], lse[last:], pool, torch.ones(1, 1, dtype=torch.int32), lens[last:], q[last:], heads, page, 0.1)
