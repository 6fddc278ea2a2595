"""The cache attention on a host without a GPU: workspace sizes and refusals,
decided before any CUDA call."""
import pytest
import torch

from tests.test_cache_host import FAKE, POOL, STREAM, Recorder, call, fake


@pytest.fixture(scope="module")
def S():
    from lossless_kv_cache_bf16_gb300 import splitzip

    return splitzip


ATTEND = dict(q=FAKE, qs=1024, qh=128, batch=2, hq=8, pool=FAKE, pages=9, heads=2, dim=128, page=16, table=FAKE,
              width=4, lens=FAKE, scale=0.1, out=2 * FAKE, os=1024, oh=128, lse=None, weight=None, status=None, ws=FAKE,
              ws_bytes=1 << 40, stream=None)


def test_workspace_sizes(S):
    size = S.sz_cache_attend_workspace_size
    assert size(1, 8, 8, 128, 4096) > 0 and size(0, 8, 8, 128, 4096) > 0
    assert size(4, 28, 4, 128, 4096, True) - size(4, 28, 4, 128, 4096) >= 4 * 28 * 4 * 4097
    for bad in ((2049, 8, 8, 128, 64), (1, 9, 8, 128, 64), (1, 8, 8, 96, 64), (1, 0, 8, 128, 64), (1, 8, 0, 128, 64),
                (1, 8, 8, 128, 0), (1, 8, 8, 128, 1 << 31), (1, 2048, 1, 128, 64)):
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("change", POOL + [
    dict(batch=2049), dict(hq=9), dict(hq=0), dict(hq=4096), dict(table=None), dict(table=FAKE + 2), dict(width=0),
    dict(width=1 << 27), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(out=None),
    dict(q=FAKE + 1), dict(lens=None), dict(lens=FAKE + 2), dict(lse=FAKE + 2), dict(weight=FAKE + 2),
    dict(ws=None), dict(ws=FAKE + 16), dict(status=FAKE + 2)], ids=str)
def test_bad_arguments_are_refused_before_any_launch(S, change):
    assert call(S.LIB, "sz_cache_attend", ATTEND, **change) == S.SZ_ERR_INVALID_ARG


def test_nothing_to_do_launches_nothing(S):
    assert call(S.LIB, "sz_cache_attend", ATTEND, batch=0, q=None, out=None, lens=None, table=None, ws=None) == S.SZ_OK


def test_binding_refuses_mismatched_tensors(S, monkeypatch):
    rec = Recorder(S._bind)
    monkeypatch.setattr(S, "_bind", rec)
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    t = fake
    pool = t(9, S.sz_cache_page_bytes(128, 2, 16), dtype=u8)
    cells = 9 * 2 * 16
    q = t(4, 8, 128)
    out = t(4, 8, 128)
    out.data_ptr = lambda: 2 * FAKE
    attend = lambda **c: S.sz_cache_attend(**{**dict(q=q, pool=pool, kv_heads=2, page_tokens=16,
                                                     table=t(4, 3, dtype=i32), lens=t(4, dtype=i32), scale=0.1, out=out,
                                                     ws=t(8, dtype=u8), stream=STREAM), **c})
    attend()
    assert rec.calls == ["cache_attend"]
    del rec.calls[:]
    for c in (dict(out=t(4, 8, 64)), dict(out=q), dict(table=t(3, 3, dtype=i32)), dict(table=t(4, 3, dtype=torch.int64)),
              dict(table=t(12, dtype=i32)), dict(table=t(4, 6, dtype=i32)[:, ::2]), dict(lens=t(3, dtype=i32)),
              dict(lse=t(31, dtype=f32)), dict(weight=t(cells + 1, dtype=f32)), dict(out=t(1, 8, 128).expand(4, 8, 128)),
              dict(status=t(1, dtype=torch.int64)), dict(q=t(4, 8, 128, dtype=f32)),
              dict(pool=torch.empty(9, 4608, dtype=u8))):
        with pytest.raises(ValueError):
            attend(**c)
    assert rec.calls == []
