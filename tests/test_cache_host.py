"""The serving operators on a host without a GPU: page sizes, workspace sizes
and refusals, all decided before any CUDA call.  No compute runs here."""
import ctypes
import re

import pytest
import torch

from tests import cache_ref as R
from tests.test_abi import HEADER

FAKE = 0x10000


@pytest.fixture(scope="module")
def S():
    from lossless_kv_cache_bf16_gb300 import splitzip

    return splitzip


def test_page_bytes(S):
    for dim in (64, 128):
        for heads in (1, 3, 8):
            for page in (16, 64, 4096):
                assert S.sz_cache_page_bytes(dim, heads, page) == R.page_bytes(dim, heads, page)
    for bad in ((96, 8, 64), (256, 8, 64), (128, 0, 64), (128, 4097, 64), (128, 8, 8), (128, 8, 48), (128, 8, 8192)):
        assert S.sz_cache_page_bytes(*bad) == 0


def test_cell_words_are_a_permutation():
    """Every word of a cell belongs to one token; 16 tokens fill it."""
    for dim in (64, 128):
        for first in (0, 16):
            seen = [w for t in range(16) for part in R.words_of_token(dim, first + t) for w in part]
            assert sorted(seen) == list(range(first // 16 * 9 * dim, (first // 16 + 1) * 9 * dim))


def test_reference_quantisation():
    """Hand-worked group: max 3.5, scale 0.5, ties to even, -0 and 0 alike."""
    x = torch.zeros(32, dtype=torch.bfloat16)
    x[:8] = torch.tensor([3.5, -3.5, 0.25, 0.75, -0.25, -0.75, 1.25, -0.0])
    codes, s = R.quantise(x)
    assert s.tolist() == [0.5]
    assert codes[:9].tolist() == [15, 1, 8, 10, 8, 6, 10, 8, 8]
    x[3] = float("inf")
    codes, s = R.quantise(x)
    assert torch.isnan(s).all() and (codes == 8).all()
    codes, s = R.quantise(torch.full((32,), 2.0 ** -126, dtype=torch.bfloat16))
    assert s.tolist() == [0.0] and (codes == 8).all()


def test_workspace_sizes(S):
    assert S.sz_cache_evict_workspace_size(2, 8, 1000) >= 2 * 8 * (4 + 8 * 500)
    for bad in ((65536, 8, 64), (1, 0, 64), (1, 8, 0), (1, 8, 1 << 31)):
        assert S.sz_cache_evict_workspace_size(*bad) == 0


def call(lib, name, defaults, **change):
    args = dict(defaults)
    for k in change:
        assert k in args, k
    args.update(change)
    return getattr(lib, name)(*args.values())


NORM = dict(q=FAKE, qt=1024, qh=128, hq=8, k=FAKE, kt=1024, kh=128, hk=2, tokens=4, dim=128, wq=FAKE, wk=FAKE,
            eps=1e-6, freq=FAKE, rot=128, inter=0, positions=FAKE, qo=FAKE, qot=1024, qoh=128, ko=FAKE, kot=1024,
            koh=128, stream=None)
APPEND = dict(k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, tokens=4, slots=FAKE, positions=None, pool=FAKE, pages=9,
              heads=2, dim=128, page=16, weight=None, pos=None, status=None, stream=None)
READ = dict(pool=FAKE, pages=9, heads=2, dim=128, page=16, slots=FAKE, tokens=4, k=FAKE, kt=256, kh=128, v=FAKE,
            vt=256, vh=128, status=None, stream=None)
EVICT = dict(pool=FAKE, pages=9, heads=2, dim=128, page=16, table=FAKE, width=4, lens=FAKE, nxt=FAKE, batch=2, keep=8,
             recent=2, weight=FAKE, pos=FAKE, new=2 * FAKE, status=None, ws=FAKE, ws_bytes=1 << 40, stream=None)

POOL = [dict(pool=None), dict(pool=FAKE + 8), dict(pages=0), dict(pages=1 << 31), dict(heads=0), dict(dim=96),
        dict(page=8), dict(page=24), dict(page=8192)]


@pytest.mark.parametrize("name,defaults,changes", [
    ("sz_qk_norm_rope", NORM, [
        dict(dim=96), dict(hq=0, hk=0), dict(hq=65537), dict(tokens=1 << 31), dict(rot=144), dict(rot=24),
        dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(freq=None), dict(freq=FAKE + 2),
        dict(positions=None), dict(positions=FAKE + 1), dict(q=None), dict(q=FAKE + 1), dict(k=None), dict(qo=None),
        dict(ko=FAKE + 1), dict(wq=FAKE + 1)]),
    ("sz_cache_append", APPEND, POOL + [
        dict(tokens=1 << 31), dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(slots=None), dict(slots=FAKE + 4),
        dict(pos=FAKE), dict(pos=FAKE + 2, positions=FAKE), dict(weight=FAKE + 2), dict(status=FAKE + 2)]),
    ("sz_cache_read", READ, POOL + [
        dict(tokens=1 << 31), dict(k=None), dict(v=FAKE + 1), dict(slots=None), dict(slots=FAKE + 4),
        dict(status=FAKE + 1)]),
    ("sz_cache_evict", EVICT, POOL + [
        dict(batch=65536), dict(keep=0), dict(keep=1 << 31), dict(recent=1 << 31), dict(table=None), dict(width=0),
        dict(lens=None), dict(nxt=None), dict(new=None), dict(new=FAKE), dict(weight=None), dict(pos=None),
        dict(pos=FAKE + 2), dict(ws=None), dict(ws=FAKE + 4), dict(status=FAKE + 2)]),
])
def test_bad_arguments_are_refused_before_any_launch(S, name, defaults, changes):
    for change in changes:
        assert call(S.LIB, name, defaults, **change) == S.SZ_ERR_INVALID_ARG, change


def test_small_workspace_is_refused(S):
    assert call(S.LIB, "sz_cache_evict", EVICT, ws_bytes=S.sz_cache_evict_workspace_size(2, 2, 64) - 1) == S.SZ_ERR_CAPACITY


def test_nothing_to_do_launches_nothing(S):
    assert call(S.LIB, "sz_qk_norm_rope", NORM, tokens=0, q=None, k=None, positions=None) == S.SZ_OK
    assert call(S.LIB, "sz_cache_append", APPEND, tokens=0, k=None, v=None, slots=None) == S.SZ_OK
    assert call(S.LIB, "sz_cache_read", READ, tokens=0, k=None, v=None, slots=None) == S.SZ_OK
    assert call(S.LIB, "sz_cache_evict", EVICT, batch=0, lens=None, nxt=None, new=None) == S.SZ_OK


class Cuda(torch.Tensor):
    """A tensor without storage that says it is on the GPU."""
    is_cuda = True

    def data_ptr(self):
        return FAKE


def fake(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(Cuda)


class Recorder:
    """Stands for the binding's C++ part: checks tensors as it does and records
    the calls that would launch."""

    def __init__(self, bind):
        self.rows, self.written_rows, self.pointer, self.calls = bind.rows, bind.written_rows, bind.pointer, []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


STREAM = type("Stream", (), {"cuda_stream": 0})()


def test_binding_refuses_mismatched_tensors(S, monkeypatch):
    """Shapes, types and sizes that would let a kernel leave a buffer are
    refused by the binding; the library is not called."""
    rec = Recorder(S._bind)
    monkeypatch.setattr(S, "_bind", rec)
    i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8
    t, s = fake, STREAM
    q, k = t(4, 8, 128), t(4, 2, 128)
    freq, position = t(64, dtype=f32), t(4, dtype=i32)
    norm = lambda **c: S.sz_qk_norm_rope(**{**dict(q=q, k=k, q_weight=t(128), k_weight=t(128), eps=1e-6, inv_freq=freq,
                                                   positions=position, q_out=t(4, 8, 128), k_out=t(4, 2, 128),
                                                   stream=s), **c})
    pool = t(9, S.sz_cache_page_bytes(128, 2, 16), dtype=u8)
    cells = 9 * 2 * 16
    append = lambda **c: S.sz_cache_append(**{**dict(k=k, v=t(4, 2, 128), slots=t(4, dtype=i64), pool=pool,
                                                     page_tokens=16, stream=s), **c})
    read = lambda **c: S.sz_cache_read(**{**dict(pool=pool, page_tokens=16, slots=t(4, dtype=i64), k=k,
                                                 v=t(4, 2, 128), stream=s), **c})
    evict = lambda **c: S.sz_cache_evict(**{**dict(pool=pool, kv_heads=2, head_dim=128, page_tokens=16,
                                                   table=t(4, 3, dtype=i32), lens=t(4, dtype=i32),
                                                   next_pos=t(4, dtype=i32), keep=8, recent=2,
                                                   weight=t(cells, dtype=f32), pos=t(cells, dtype=i32),
                                                   new_lens=t(4, dtype=i32), ws=t(8, dtype=u8), stream=s), **c})
    for f in (norm, append, read, evict):
        f()
    assert len(rec.calls) == 4
    del rec.calls[:]
    bad = [
        (norm, dict(q=t(4, 8, 128, dtype=f32))), (norm, dict(k=t(3, 2, 128))), (norm, dict(k=t(4, 2, 64))),
        (norm, dict(q=t(4, 1024))), (norm, dict(q_out=t(4, 8, 64))), (norm, dict(q_weight=t(64))),
        (norm, dict(k_weight=t(128, dtype=f32))), (norm, dict(positions=t(4, dtype=i64))),
        (norm, dict(positions=t(3, dtype=i32))), (norm, dict(inv_freq=t(64))),
        (norm, dict(q_out=t(4, 1, 128).expand(4, 8, 128))), (norm, dict(q=t(8, 4, 128).transpose(0, 1))),
        (norm, dict(q=t(4, 8, 256)[:, :, ::2])), (norm, dict(q=torch.empty(4, 8, 128, dtype=torch.bfloat16))),
        (append, dict(v=t(4, 2, 64))), (append, dict(slots=t(4, dtype=i32))), (append, dict(slots=t(5, dtype=i64))),
        (append, dict(weight=t(cells - 1, dtype=f32))), (append, dict(pos=t(cells, dtype=i32))),
        (append, dict(pos=t(cells - 1, dtype=i32), positions=position)), (append, dict(status=t(2, dtype=i32))),
        (append, dict(pool=t(9, 64, dtype=u8)[:, ::2])), (append, dict(page_tokens=-16)),
        (read, dict(v=t(4, 3, 128))), (read, dict(slots=t(3, dtype=i64))), (read, dict(k=t(4, 1, 128).expand(4, 2, 128))),
        (evict, dict(weight=t(cells, dtype=torch.float64))), (evict, dict(pos=t(cells - 1, dtype=i32))),
        (evict, dict(next_pos=t(3, dtype=i32))), (evict, dict(new_lens=t(3, dtype=i32))), (evict, dict(keep=-1)),
        (evict, dict(recent=-1)), (evict, dict(table=t(2, 3, dtype=i32))),
    ]
    for f, c in bad:
        with pytest.raises(ValueError):
            f(**c)
    assert rec.calls == []


def test_overlapping_outputs(S):
    """Rows that share memory are told from rows that interleave."""
    b = S._bind
    ok = [fake(4, 2, 64), fake(2, 4, 64).transpose(0, 1), fake(4, 6, 64)[:, 2:4], fake(4, 2, 70)[..., :64],
          fake(1, 1, 64).expand(1, 1, 64), fake(0, 2, 64), fake(4, 1, 64)[:, :1]]
    for t in ok:
        assert b.written_rows(t, torch.bfloat16, t.shape, "t")[1:] == (t.shape, t.stride())
    for t in (fake(1, 2, 64).expand(4, 2, 64), fake(4, 1, 64).expand(4, 2, 64), fake(600).as_strided((4, 2, 64), (64, 32, 1)),
              fake(600).as_strided((4, 2, 64), (64, 64, 1)), fake(600).as_strided((2, 4, 64), (100, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            b.written_rows(t, torch.bfloat16, t.shape, "t")
    with pytest.raises(ValueError, match="shape"):
        b.written_rows(ok[0], torch.bfloat16, (4, 2, 32), "t")


def test_bad_values_do_not_reach_the_library(S):
    """Python values that are no numbers of the right kind raise; the call is
    not made (address 0 would end the process if it were)."""
    ok = [0, *APPEND.values()]
    for at, bad in ((1, "x"), (2, 1.5), (7, -1), (7, None), (15, object()), (18, "stream")):
        args = list(ok)
        args[at] = bad
        with pytest.raises((TypeError, OverflowError, ValueError)):
            S._bind.cache_append(*args)
    with pytest.raises(TypeError):
        S._bind.cache_append(*ok[:-1])
    with pytest.raises(ValueError):
        S._bind.cache_append(*ok)
    good = [S._ADDRESS["sz_cache_append"], *APPEND.values()]
    good[7] = 0                                              # no tokens: nothing is launched
    assert S._bind.cache_append(*good) == S.SZ_OK
    good[10] = None
    assert S._bind.cache_append(*good) == S.SZ_ERR_INVALID_ARG
    for name, defaults in (("qk_norm_rope", NORM), ("cache_read", READ), ("cache_evict", EVICT)):
        args = [S._ADDRESS["sz_" + name], *defaults.values()]
        args[1 + list(defaults).index("dim")] = 96
        assert getattr(S._bind, name)(*args) == S.SZ_ERR_INVALID_ARG
    # A float argument arrives: a negative eps is refused, a good one passes.
    args = [S._ADDRESS["sz_qk_norm_rope"], *{**NORM, "tokens": 0}.values()]
    assert S._bind.qk_norm_rope(*args) == S.SZ_OK
    args[1 + list(NORM).index("eps")] = -1.0
    assert S._bind.qk_norm_rope(*args) == S.SZ_ERR_INVALID_ARG


def test_signatures_cover_the_declared_arguments(S):
    """The ctypes signatures have the header's arguments, by number and kind."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = [n for n in re.findall(r"\b(sz_[a-z_]+)\s*\(", text) if n.startswith("sz_cache_") or n == "sz_qk_norm_rope"]
    assert len(names) >= 6
    for name in names:
        args = re.search(r"\b" + name + r"\((.*?)\);", text, flags=re.S).group(1)
        assert len(args.split(",")) == len(getattr(S.LIB, name).argtypes), name
        for a, kind in zip(args.split(","), getattr(S.LIB, name).argtypes):
            want = ctypes.c_void_p if "*" in a or "cudaStream_t" in a else \
                {"size_t": ctypes.c_size_t, "int64_t": ctypes.c_int64, "int": ctypes.c_int, "float": ctypes.c_float}[a.split()[0]]
            assert kind is want, (name, a)
