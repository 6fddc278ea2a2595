"""Attention of drafted tokens where sequences have trees of different sizes:
items whose rows leave a group of softmax warps without any, among others.

Tolerances as in test_gpu_tree.py.
"""
import random

import pytest
import torch

from tests import cache_ref as R
from tests import test_gpu_tree as tree
from tests import tree_ref as T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    from lossless_kv_cache_bf16_gb300 import splitzip

    tree.S = splitzip


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,heads,group,nodes,counts", [
    ([20000, 300, 0, 9000], 1, 4, 16, [8, 16, 3, 1]), ([3000] * 6, 4, 4, 16, [1, 16, 8, 0, 9, 2]),
    ([700, 1500, 40] * 8, 2, 7, 20, [1, 20, 4, 14, 9, 5] * 4), ([50000], 1, 40, 64, [2])])
def test_few_rows_among_many(lens, heads, group, nodes, counts, dim):
    """Up to 32 rows of a sequence, and more, or a last item with few, over many tiles."""
    c = tree.Case(lens, heads, group, dim, 32, nodes, seed=31, counts=counts)
    first = c.run()
    c.check(*first)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run()))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,heads,group,nodes", [([20000], 2, 4, 4), ([9000, 30000], 1, 4, 8), ([40000], 1, 7, 64),
                                                    ([2500] * 20, 2, 4, 16)])
def test_bad_nodes_behind_long_contexts(lens, heads, group, nodes, dim):
    """Items whose last tokens are another block's than their first: a node whose
    V is not finite reaches the nodes that attend to it, in its channels."""
    c = tree.Case(lens, heads, group, dim, 32, nodes, seed=32)
    rng, n = random.Random(dim + nodes), len(lens)
    k, v = R.normal_bf16(R.gen(7), n, heads, dim), R.normal_bf16(R.gen(8), n, heads, dim)
    want, slots = torch.zeros(n, nodes, heads * group, dim, dtype=torch.bool), []
    for b in range(n):
        node, head, channels = rng.randrange(nodes), rng.randrange(heads), rng.randrange(dim // 32)
        v[b, head, 32 * channels + 5] = float("nan") if b % 2 else -float("inf")
        slots.append(int(c.slots(b, lens[b] + nodes)[lens[b] + node]))
        want[b, (c.mask[b] >> node & 1).bool(), head * group:(head + 1) * group, 32 * channels:32 * channels + 32] = True
    c.write(k, v, torch.tensor(slots))
    for _ in range(10):
        out, lse = c.run()
        assert torch.equal(torch.isnan(out).cpu(), want) and not bool(torch.isnan(lse).any())


@pytest.mark.parametrize("group,counts", [(4, range(1, 17)), (8, range(1, 17)), (4, [16, 4, 4, 4]), (10, [16, 13, 0, 1])])
@pytest.mark.parametrize("dim", [64, 128])
def test_bad_nodes_stay_in_their_sequence(dim, group, counts):
    """Blocks with many items of one tile, some of few rows and some of many: a node
    whose V is not finite reaches the nodes of its sequence that attend to it,
    and no row of another one."""
    rng, n, nodes = random.Random(dim + group), 1500, 16
    counts = [rng.choice(list(counts)) for _ in range(n)]
    c = tree.Case([rng.randrange(0, 100) for _ in range(n)], 1, group, dim, 16, nodes, seed=33, counts=counts)
    bad = [b for b in range(n) if counts[b] and rng.random() < 0.4]
    k, v = R.normal_bf16(R.gen(7), len(bad), 1, dim), R.normal_bf16(R.gen(8), len(bad), 1, dim)
    want = torch.zeros(n, nodes, group, dim, dtype=torch.bool)
    slots = []
    for at, b in enumerate(bad):
        # Roots most often, which every node attends to.
        node, channels = 0 if rng.random() < 0.7 else rng.randrange(counts[b]), rng.randrange(dim // 32)
        v[at, 0, 32 * channels + at % 32] = float("nan") if at % 2 else float("inf")
        slots.append(int(c.slots(b, c.lens[b] + counts[b])[c.lens[b] + node]))
        sees = (c.mask[b] >> node & 1).bool() & (torch.arange(nodes) < counts[b])
        want[b, sees, :, 32 * channels:32 * channels + 32] = True
    c.write(k, v, torch.tensor(slots))
    for _ in range(3):
        out, _ = c.run()
        assert torch.equal(torch.isnan(out).cpu(), want)


def test_rows_of_a_wide_sequence_that_cannot_be_served():
    """2^32 outputs of a sequence with a negative length: all zero."""
    S, nodes, heads, group, dim = tree.S, 64, 512, 1024, 128
    hq = heads * group
    pool = torch.zeros(1, R.page_bytes(dim, heads, 16), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = torch.full((1, nodes, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    lse, status = torch.full((1, nodes, hq), 7.0, device="cuda"), i32([-1])
    ws = torch.empty(S.sz_cache_attend_tree_workspace_size(1, nodes, hq, heads, dim, 16), dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 1, 1, dim, dtype=torch.bfloat16, device="cuda").expand(1, nodes, hq, dim)
    S.sz_cache_attend_tree(q, pool, heads, 16, i32([[0]]), i32([-1]), torch.ones(1, nodes, dtype=torch.int64, device="cuda"), 0.1, out, ws,
                           lse=lse, status=status)
    assert status.item() == S.SZ_ERR_INVALID_ARG
    assert all(bool((out[0, j] == 0).all()) for j in range(nodes)) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("nodes,group", [(2, 1), (8, 4), (16, 4)])
def test_rows_that_share_a_power_of_two(nodes, group):
    """Every other row 2^-12 of its neighbours, its logits from a channel 2^-26 of
    its largest: they are good to 2^-27 of a row's largest value in each channel."""
    c = tree.Case([100], 1, group, 64, 16, nodes, seed=35)
    c.scale = 0.125
    k = torch.zeros(100 + nodes, 1, 64)
    k[:, 0, 1] = 2.0 ** 38 * (1 + torch.arange(100 + nodes) % 7)
    c.write(k.to(torch.bfloat16), R.normal_bf16(R.gen(9), 100 + nodes, 1, 64), c.slots(0, 100 + nodes))
    c.q[:] = 0
    c.q[:, ::2, :, 0] = 1.0
    c.q[:, 1::2, :, 0] = 2.0 ** -12
    small = torch.arange(nodes * group).view(nodes, group)[1::2] % 16
    c.q[0, 1::2, :, 1] = (2.0 ** -38 * (0.25 + small / 8)).to(torch.bfloat16)
    out, lse = c.run()
    held, v, scales = T.values(c.pool, c.slots(0, 100 + nodes), 16, 1, 64)
    assert bool((held[:, 0, 0] == 0).all()) and bool((held[:, 0, 1] >= 2.0 ** 37).all())  # the scales are rounded
    _, _, want, err = T.attend(c.q[0].cuda(), held, v, scales, c.sees(0).cuda(), c.scale)
    shared = 2.0 ** -27 * c.q[0].cuda().double().abs().amax(-1) * float(held.abs().sum(-1).max()) * c.scale
    off = (lse[0].double() - want).abs()
    assert bool((off <= err + shared + 2.0 ** -18 * (1 + want.abs())).all())


@pytest.mark.parametrize("bad", [0x7F7F, -0x0081, 0x7F70])
@pytest.mark.parametrize("dim,nodes,group", [(64, 4, 4), (128, 6, 4), (128, 16, 8)])
def test_a_node_of_the_largest_values(dim, nodes, group, bad):
    """V of the largest bf16 numbers, which the cache holds as more than that: rows
    that do not attend to the node are as if it held zero, and no row is NaN."""
    big = float(torch.tensor([bad], dtype=torch.int16).view(torch.bfloat16)[0])
    c = tree.Case([30, 0, 125, 127], 2, group, dim, 16, nodes, seed=36)
    k, v = R.normal_bf16(R.gen(7), 1, 2, dim), torch.zeros(1, 2, dim, dtype=torch.bfloat16)
    outs = []
    for value in (0.0, big):
        v[0, :, 5], v[0, :, 37] = value, -value
        for b, n in enumerate(c.lens):
            c.write(k, v, c.slots(b, n + nodes)[n + 2:n + 3])
        outs.append(c.run())
    sees = (c.mask >> 2 & 1).bool()
    assert bool(sees.any()) and not bool(sees.all())
    assert not bool(torch.isnan(outs[1][0]).any()) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(outs[0][0][~sees], outs[1][0][~sees])


@pytest.mark.parametrize("lens,counts", [([20000, 300, 9000], [8, 16, 3]), ([40] * 400, [1, 16, 8, 12] * 100)])
def test_a_wait_that_gives_up_beside_few_rows(lens, counts):
    """As in test_gpu_tree.py, with items that have no rows for some warps."""
    c = tree.Case(lens, 1, 4, 128, 64, 16, seed=37, counts=counts)
    want = c.run()
    S, (b, n, hq, d) = tree.S, c.q.shape
    ws = torch.empty(S.sz_cache_attend_tree_workspace_size(b, n, hq, 1, d, c.table.shape[1] * 64), dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    S.sz_debug_attend_tree_stalled(c.q.cuda(), c.pool, 1, 64, c.table.cuda(), i32(lens), c.mask.cuda(), c.scale, out, ws, counts=i32(counts),
                                   lse=lse, status=status)
    assert status.item() == S.SZ_ERR_TIMEOUT
    lost = torch.isnan(out).all(-1)
    assert bool(lost[0, :counts[0]].all()) and bool((torch.isnan(lse) == lost).all())
    assert torch.equal(out[~lost], want[0][~lost])
    assert all(torch.equal(x, y) for x, y in zip(c.run(), want))
