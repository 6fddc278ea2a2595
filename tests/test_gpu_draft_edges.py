"""Drafts near the end of a DecodeCache."""
import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32)])
def test_a_full_sequence_and_one_with_room(dim, page):
    """As in a larger cache; the full sequence's tokens stay as they are."""
    from lossless_kv_cache_bf16_gb300 import decode, splitzip as S

    hk, hq, nodes, g = 2, 8, 6, R.gen(dim)
    caches = [decode.DecodeCache(2, hq, hk, dim, n, page_tokens=page) for n in (64, 128)]
    for b, n in ((0, 64), (1, 61)):
        k, v = R.normal_bf16(g, n, hk, dim).cuda(), R.normal_bf16(g, n, hk, dim).cuda()
        for c in caches:
            c.extend(b, k, v)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(dim // 2) * 2.0 / dim)).float().cuda()
    parents, counts = i32([[0, 0, 1, 1, 2, 0]] * 2), i32([0, 3])
    qkv = R.normal_bf16(g, 2, nodes, hq + 2 * hk, dim).cuda()
    first = caches[0].pool.clone()
    outs = []
    for c in caches:
        out = torch.full((2, nodes, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        c.draft(qkv.clone(), parents, None, None, freq, counts=counts, out=out)
        c.check()
        outs.append(out)
    assert torch.equal(*outs) and bool((outs[0][0] == 7).all()) and bool((outs[0][1, 3:] == 7).all())
    pages = 64 // page
    assert torch.equal(caches[0].pool[:pages], first[:pages])
    for c in caches:
        c.accept(i32([[-1] * 6, [0, 2] + [-1] * 4]), i32([0, 2]))
        c.check()
        assert c.held == [64, 63]
    own = [c.pool.view(2, -1, c.pool.shape[1])[:, :pages] for c in caches]
    assert torch.equal(own[0][0], own[1][0])
    # Nodes that do not fit: rows of zero, reported, nothing outside written.
    before = caches[0].pool.clone()
    out = caches[0].draft(qkv.clone(), parents, None, None, freq, counts=i32([1, 2]))
    with pytest.raises(S.SplitZipError):
        caches[0].check()
    assert bool((out[0, 0] == 0).all()) and bool((out[1, :2] == 0).all())
    assert torch.equal(caches[0].pool[:pages], before[:pages])
    caches[0].accept(i32([[0] + [-1] * 5, [0, 1] + [-1] * 4]), i32([1, 2]))
    assert caches[0].held == [64, 63]
