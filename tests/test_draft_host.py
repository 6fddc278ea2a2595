"""DecodeCache's drafts on a host without a GPU: slots near the end of a cache, and
what refused calls leave."""
import pytest
import torch

bf16 = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
i32 = lambda x: torch.tensor(x, dtype=torch.int32)


@pytest.fixture
def cache(monkeypatch):
    """A cache of 2 x 64 tokens without a GPU, whose appended slots are recorded."""
    from lossless_kv_cache_bf16_gb300 import decode

    slots = []
    for name in ("sz_qk_norm_rope", "sz_cache_attend", "sz_cache_attend_tree", "check_output"):
        monkeypatch.setattr(decode.S, name, lambda *a, **k: None)
    monkeypatch.setattr(decode.S, "sz_cache_append", lambda k, v, s, *a, **kw: slots.append(s.tolist()))

    def accept(pool, heads, dim, page, table, lens, path, accepted, new_lens, **_):
        new_lens.copy_(lens + accepted)

    monkeypatch.setattr(decode.S, "sz_cache_accept", accept)
    cache = decode.DecodeCache(2, 4, 2, 64, 64, page_tokens=16, device="cpu")
    cache.slots = slots
    return cache


def test_drafts_at_the_end_of_a_cache(cache):
    freq, parents = torch.ones(32), i32([[0, 0, 1], [0, 0, 0]])
    cache.extend(0, bf16(64, 2, 64), bf16(64, 2, 64))
    cache.extend(1, bf16(62, 2, 64), bf16(62, 2, 64))
    del cache.slots[:]
    with pytest.raises(ValueError, match="full"):
        cache.draft(bf16(2, 3, 8, 64), parents, None, None, freq)
    assert cache.slots == [] and not cache.drafted
    # None of the full one, two of the other; counts that do not fit reach no slot outside.
    for counts, want in (([0, 2], [-1] * 3 + [126, 127, -1]), ([3, 3], [-1] * 3 + [126, 127, -1]), ([0, 1], [-1] * 3 + [126, -1, -1])):
        out = cache.draft(bf16(2, 3, 8, 64), parents, None, None, freq, counts=i32(counts))
        assert out.shape == (2, 3, 4, 64) and cache.slots == [want] and cache.drafted == 3
        del cache.slots[:]
    cache.accept(i32([[-1] * 3, [0, -1, -1]]), i32([0, 1]))
    assert cache.held == [64, 63] == cache.next_pos.tolist()


def test_counts_do_not_matter_to_slots_where_there_is_room(cache):
    cache.extend(0, bf16(50, 2, 64), bf16(50, 2, 64))
    del cache.slots[:]
    for counts in (None, i32([3, 1])):
        cache.draft(bf16(2, 3, 8, 64), i32([[0, 0, 1], [0, 0, 0]]), None, None, torch.ones(32), counts=counts)
    assert cache.slots == [[50, 51, 52, 64, 65, 66]] * 2


def test_a_refused_prompt_or_step_leaves_the_draft(cache, monkeypatch):
    from lossless_kv_cache_bf16_gb300 import decode

    freq = torch.ones(32)
    cache.extend(0, bf16(5, 2, 64), bf16(5, 2, 64))
    cache.draft(bf16(2, 3, 8, 64), i32([[0, 0, 1], [0, 0, 0]]), None, None, freq)

    def refuse(*_, **__):
        raise ValueError("refused")

    with monkeypatch.context() as m:
        m.setattr(decode.S, "sz_cache_append", refuse)
        for call in (lambda: cache.extend(1, bf16(2, 2, 64).float(), bf16(2, 2, 64).float()),
                     lambda: cache.step(bf16(2, 8, 64), None, None, freq)):
            with pytest.raises(ValueError, match="refused"):
                call()
        m.setattr(decode.S, "sz_qk_norm_rope", refuse)
        with pytest.raises(ValueError, match="refused"):
            cache.step(bf16(2, 8, 64), None, None, freq)
    assert cache.held == [5, 0] == cache.lens.tolist() == cache.next_pos.tolist()
    cache.accept(i32([[0, 1, -1], [0, -1, -1]]), i32([2, 1]))
    assert cache.held == [7, 1]


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.0 ** 127 * (1 + 2.0 ** -23)])
def test_scales_beyond_what_a_product_with_log2_e_holds_are_refused(scale):
    from lossless_kv_cache_bf16_gb300 import splitzip as S
    from tests.test_cache_host import call
    from tests.test_tree_host import TREE

    assert call(S.LIB, "sz_cache_attend_tree", TREE, scale=scale, ws_bytes=0) == S.SZ_ERR_INVALID_ARG
    assert call(S.LIB, "sz_cache_attend_tree", TREE, scale=-2.0 ** 127, ws_bytes=0) != S.SZ_ERR_INVALID_ARG
