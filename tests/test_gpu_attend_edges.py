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
