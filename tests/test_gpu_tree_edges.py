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
