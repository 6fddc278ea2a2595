"""The serving operators on a host without a GPU: what their binding and the
library refuse before anything is launched."""
import random

import pytest
import torch

from tests.test_attend_host import ATTEND
from tests.test_cache_host import EVICT, FAKE, NORM, POOL, READ, Recorder, call


@pytest.fixture(scope="module")
def S():
    from lossless_kv_cache_bf16_gb300 import splitzip

    return splitzip


@pytest.mark.parametrize("change", POOL + [dict(status=None), dict(q=None), dict(ws=None), dict(hq=9)], ids=str)
def test_the_stalled_attention_refuses_what_the_attention_does(S, change):
    stalled = {**ATTEND, "status": ATTEND["lens"]}
    assert call(S.LIB, "sz_debug_attend_stalled", stalled, **change) == S.SZ_ERR_INVALID_ARG


class OnGpu(torch.Tensor):
    """A tensor without storage that says it is on the GPU of that number."""
    is_cuda = True
    gpu = 0

    def data_ptr(self):
        return FAKE

    def get_device(self):
        return self.gpu


def on_gpu(*shape, dtype=torch.bfloat16, gpu=0):
    t = torch.empty(*shape, dtype=dtype, device="meta").as_subclass(OnGpu)
    t.gpu = gpu
    return t


def stream(gpu):
    return type("Stream", (), {"cuda_stream": 0, "device_index": gpu})()


def calls(S):
    """Every operator's tensor arguments and a call with them."""
    i32, i64, f32, u8 = torch.int32, torch.int64, torch.float32, torch.uint8
    t = on_gpu
    out = t(4, 8, 128)
    out.data_ptr = lambda: 2 * FAKE
    pool, cells = t(9, S.sz_cache_page_bytes(128, 2, 16), dtype=u8), (9, 2, 16)
    norm = dict(q=t(4, 8, 128), k=t(4, 2, 128), q_weight=t(128), k_weight=t(128), inv_freq=t(64, dtype=f32),
                positions=t(4, dtype=i32), q_out=t(4, 8, 128), k_out=t(4, 2, 128))
    rows = dict(k=t(4, 2, 128), v=t(4, 2, 128), slots=t(4, dtype=i64), pool=pool, status=t(1, dtype=i32))
    tables = dict(weight=t(*cells, dtype=f32), pos=t(*cells, dtype=i32))
    append = {**rows, **tables, "positions": t(4, dtype=i32)}
    lists = dict(pool=pool, table=t(4, 3, dtype=i32), lens=t(4, dtype=i32), ws=t(8, dtype=u8), status=t(1, dtype=i32))
    attend = {**lists, "q": t(4, 8, 128), "out": out, "lse": t(4, 8, dtype=f32), "weight": tables["weight"]}
    evict = {**lists, **tables, "next_pos": t(4, dtype=i32), "new_lens": t(4, dtype=i32)}
    return [(norm, lambda **a: S.sz_qk_norm_rope(eps=1e-6, **a)), (append, lambda **a: S.sz_cache_append(page_tokens=16, **a)),
            (rows, lambda **a: S.sz_cache_read(page_tokens=16, **a)),
            (attend, lambda **a: S.sz_cache_attend(kv_heads=2, page_tokens=16, scale=0.1, **a)),
            (evict, lambda **a: S.sz_cache_evict(kv_heads=2, head_dim=128, page_tokens=16, keep=8, recent=2, **a))]


def test_tensors_of_another_gpu_are_refused(S, monkeypatch):
    """A kernel runs on the current GPU and would follow a pointer into another
    one; no call is made with such a tensor, nor on another GPU's stream."""
    rec = Recorder(S._bind)
    monkeypatch.setattr(S, "_bind", rec)
    current = 0
    monkeypatch.setattr(S.torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(S, "_get_device", lambda: current)
    monkeypatch.setattr(S, "_raw_stream", lambda device: 1000 + device)
    for args, f in calls(S):
        for given in (None, stream(0)):
            f(**args, stream=given)
        assert len(rec.calls) == 2
        del rec.calls[:]
        for name, t in args.items():
            for given in (None, stream(0)):
                other = t.as_subclass(OnGpu)
                other.gpu = 1
                other.data_ptr = t.data_ptr
                with pytest.raises(ValueError, match=name + ".* GPU"):
                    f(**{**args, name: other}, stream=given)
                other.gpu = -1
                with pytest.raises(ValueError, match=name):
                    f(**{**args, name: other}, stream=given)
        with pytest.raises(ValueError, match="stream"):
            f(**args, stream=stream(1))
        current = 1
        with pytest.raises(ValueError, match="GPU"):
            f(**args, stream=None)
        current = 0
        assert rec.calls == []


def test_a_cache_runs_on_its_own_gpu(S, monkeypatch):
    """Every method of a DecodeCache makes the cache's GPU the current one."""
    from lossless_kv_cache_bf16_gb300 import decode

    current, used = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()

    for name in ("sz_qk_norm_rope", "sz_cache_append", "sz_cache_attend", "sz_cache_evict", "sz_decode"):
        monkeypatch.setattr(decode.S, name, lambda *a, name=name, **k: used.append((name, current[-1])))
    monkeypatch.setattr(decode.torch.cuda, "device", Device)
    cache = decode.DecodeCache(1, 4, 2, 64, 64, page_tokens=16, budget=16, device="cpu")
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    gpu1 = type("Gpu", (), {"type": "cuda", "index": 1})()
    cache._gpu = lambda: Device(gpu1)
    cache.extend(0, rows, rows)
    cache.extend_from_stream(0, torch.zeros(8, dtype=torch.uint8), 8, 2)
    for _ in range(40):
        cache.step(torch.zeros(1, 8, 64, dtype=torch.bfloat16), None, None, torch.ones(32))
    assert {name for name, _ in used} == {"sz_qk_norm_rope", "sz_cache_append", "sz_cache_attend", "sz_cache_evict", "sz_decode"}
    assert {gpu for _, gpu in used} == {1} and current == [0]
    with pytest.raises(ValueError, match="GPU"):
        cache.extend_from_stream(0, torch.zeros(8, dtype=torch.uint8, device="meta"), 8, 2)
    cache = decode.DecodeCache(1, 4, 2, 64, 64, page_tokens=16, device="cpu")
    cache.device = torch.device("cuda:1")
    assert cache._gpu().index == 1


def test_rows_of_another_head_count_than_the_pools_are_refused(S, monkeypatch):
    """A pool's bytes make whole pages for other head counts and page sizes
    too; its shape, and the tables', say which ones are meant."""
    rec = Recorder(S._bind)
    monkeypatch.setattr(S, "_bind", rec)
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    t, pages, heads, page = on_gpu, 20, 8, 16
    size = S.sz_cache_page_bytes(128, heads, page)
    table = lambda *shape: (t(*shape, dtype=f32), t(*shape, dtype=i32))

    def append(pool, rows=heads, page=page, weight=None, pos=None):
        S.sz_cache_append(t(4, rows, 128), t(4, rows, 128), t(4, dtype=torch.int64), pool, page, positions=t(4, dtype=i32),
                          weight=weight, pos=pos, stream=stream(-1))

    weight, pos = table(pages, heads, page)
    good = [t(pages, size, dtype=u8), t(pages, heads, size // heads, dtype=u8), t(pages * size, dtype=u8),
            t(1, pages * size, dtype=u8), t(4, 5, size, dtype=u8), t(pages, size // 2), t(1, pages, size, dtype=u8)]
    for pool in good:
        append(pool)
        append(pool, weight=weight, pos=pos)
        flat = table(pages * heads * page)
        append(pool, weight=flat[0], pos=flat[1])
    assert rec.calls == ["cache_append"] * 3 * len(good)
    del rec.calls[:]
    for rows, other in ((4, page), (2, page), (16, page), (heads, 32)):
        for pool in (good[0], good[1], good[4], good[5], good[6]):
            with pytest.raises(ValueError, match="pool"):
                append(pool, rows, other)
    flat = good[2]
    for rows, other in ((4, page), (2, page), (16, page), (1, 128)):
        with pytest.raises(ValueError, match="weight"):
            append(flat, rows, other, weight=weight)
        with pytest.raises(ValueError, match="pos"):
            append(flat, rows, other, pos=pos)
    for bad in ((heads, pages, page), (pages, page, heads), (pages, heads, page + 1), (pages * heads * page + 1,)):
        weight, pos = table(*bad)
        with pytest.raises(ValueError, match="weight"):
            append(good[0], weight=weight)
        with pytest.raises(ValueError, match="pos"):
            append(good[0], pos=pos)
    assert rec.calls == []


@pytest.fixture
def cache(S, monkeypatch):
    """A DecodeCache without a GPU, whose calls are recorded."""
    from lossless_kv_cache_bf16_gb300 import decode

    made = []
    for name in ("sz_qk_norm_rope", "sz_cache_append", "sz_cache_attend", "sz_cache_evict", "sz_decode"):
        monkeypatch.setattr(decode.S, name, lambda *a, name=name, **k: made.append(name))
    cache = decode.DecodeCache(2, 4, 2, 64, 64, page_tokens=16, budget=16, recent=4, device="cpu")
    cache.calls = made
    return cache


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_a_cache_refuses_rows_that_are_not_its_own(cache):
    state = lambda: (cache.lens.tolist(), cache.next_pos.tolist(), list(cache.held))
    before = state()
    for k, v in ((bf16(3, 4, 64), bf16(3, 4, 64)), (bf16(3, 1, 64), bf16(3, 1, 64)), (bf16(3, 2, 128), bf16(3, 2, 128)),
                 (bf16(3, 2, 64), bf16(4, 2, 64)), (bf16(3, 2, 64), bf16(3, 1, 64)), (bf16(6, 64), bf16(6, 64))):
        with pytest.raises(ValueError):
            cache.extend(0, k, v)
    freq = torch.ones(32)
    for qkv in (bf16(2, 7, 64), bf16(1, 8, 64), bf16(2, 8, 128), bf16(2, 512), bf16(2, 12, 64)):
        with pytest.raises(ValueError):
            cache.step(qkv, None, None, freq)
    assert cache.calls == [] and state() == before


def test_overlap_of_rows_against_every_byte(S):
    """overlap() against the sets of elements, for views of one small buffer."""
    rng = random.Random(7)
    room = torch.zeros(400, dtype=torch.bfloat16)
    found = [0, 0]
    for _ in range(4000):
        dim = rng.choice([1, 2, 8])
        strides = (rng.choice([0, 1, 3, 8, 12, 24, 40]), rng.choice([0, 1, 5, 8, 16, 48]))

        def view():
            size = (rng.randrange(0, 5), rng.randrange(0, 4), dim)
            step = (*(s if rng.random() < 0.9 else rng.choice([2, 8, 30]) for s in strides), 1)
            at = rng.randrange(0, 40)
            t = room.as_strided(size, step, at)
            hit = {at + i * step[0] + j * step[1] + c for i in range(size[0]) for j in range(size[1]) for c in range(dim)}
            return (t.data_ptr() or room.data_ptr(), size, step), hit

        (a, in_a), (b, in_b) = view(), view()
        got, want = S._bind.overlap(a, b), bool(in_a & in_b)
        assert got == S._bind.overlap(b, a)
        common = all(a[1][k] <= 1 or b[1][k] <= 1 or a[2][k] == b[2][k] for k in range(2))
        if common or want:
            assert got == want, (a, b)
            found[want] += 1
    assert min(found) > 500


def test_rows_that_share_memory_with_an_output_are_refused(S):
    """Views of one packed buffer (8 query, 2 key and 2 value heads of a token
    side by side) that lie apart, in place, and over one another."""
    at = lambda head, token=0: FAKE + 2 * 128 * (12 * token + head)
    packed = dict(qt=12 * 128, kt=12 * 128, qot=12 * 128, kot=12 * 128, q=at(0), k=at(8))
    norm = lambda **c: call(S.LIB, "sz_qk_norm_rope", {**NORM, **packed}, **c)
    for bad in (dict(qo=at(8), ko=at(8)), dict(qo=at(1), ko=at(8)), dict(qo=at(0), ko=at(7)), dict(qo=at(0), ko=at(9)),
                dict(qo=at(0, 1), ko=at(8)), dict(qo=at(0) + 2, ko=at(8)), dict(qo=at(0), ko=at(0)),
                dict(qo=at(4), ko=at(10)), dict(qo=at(0), qot=8 * 128, ko=at(8)), dict(qo=2 * FAKE, ko=2 * FAKE)):
        assert norm(**bad) == S.SZ_ERR_INVALID_ARG, bad
    read = lambda **c: call(S.LIB, "sz_cache_read", READ, **c)
    assert read(k=FAKE, v=FAKE + 2 * 128) == S.SZ_ERR_INVALID_ARG
    attend = lambda **c: call(S.LIB, "sz_cache_attend", ATTEND, **c)
    for out in (FAKE, FAKE + 256, FAKE - 256, FAKE + 2048, FAKE + 2):
        assert attend(out=out) == S.SZ_ERR_INVALID_ARG
    # What lies apart gets as far as the workspace, which is too small here.
    for change in (dict(out=FAKE + 4096), dict(qs=12 * 128, os=12 * 128, out=at(8), hq=4), dict(q=3 * FAKE)):
        assert attend(**change, ws_bytes=0) in (S.SZ_ERR_CAPACITY, S.SZ_ERR_UNSUPPORTED, S.SZ_ERR_CUDA), change


def test_new_lengths_over_what_other_blocks_still_read_are_refused(S):
    """Three sequences' lengths, each array shifted over another."""
    evict = lambda **c: call(S.LIB, "sz_cache_evict", EVICT, batch=3, **c)
    for off in (-8, -4, 0, 4, 8):
        for change in (dict(nxt=3 * FAKE, new=FAKE + off), dict(nxt=3 * FAKE, new=3 * FAKE + off)):
            assert evict(**change) == S.SZ_ERR_INVALID_ARG, change
    for change in (dict(nxt=3 * FAKE, new=FAKE + 12), dict(nxt=3 * FAKE, new=3 * FAKE - 12), dict(nxt=FAKE, new=2 * FAKE)):
        assert evict(**change, ws_bytes=0) == S.SZ_ERR_CAPACITY, change


def test_an_empty_batch_has_nothing_to_evict(S):
    """Tensors of no values have no address: none is asked for."""
    none = dict(batch=0, table=None, lens=None, nxt=None, new=None)
    assert call(S.LIB, "sz_cache_evict", EVICT, **none, ws=None, ws_bytes=0) == S.SZ_OK
    assert call(S.LIB, "sz_cache_evict", EVICT, **none, width=0) == S.SZ_OK
    for bad in (dict(pool=None), dict(weight=None), dict(keep=0), dict(status=FAKE + 2), dict(dim=96)):
        assert call(S.LIB, "sz_cache_evict", EVICT, **none, **bad) == S.SZ_ERR_INVALID_ARG


def test_in_place_strides_that_no_row_uses_may_differ(S, monkeypatch):
    """Norm and rotation in place: strides over one token, one head or none
    place no row, and empty tensors all have the same address."""
    rec = Recorder(S._bind)
    monkeypatch.setattr(S, "_bind", rec)
    view = lambda shape, strides: on_gpu(4096).as_strided(shape, strides)

    def empty(shape, strides):
        t = view(shape, strides)
        t.data_ptr = lambda: 0
        return t

    q = on_gpu(3, 4, 64)

    def norm(k, k_out, tokens=3, q=q, q_out=q):
        S.sz_qk_norm_rope(q, k, None, None, 1e-6, on_gpu(32, dtype=torch.float32), on_gpu(tokens, dtype=torch.int32), q_out,
                          k_out, stream=stream(-1))

    norm(empty((3, 0, 64), (768, 64, 1)), empty((3, 0, 64), (0, 64, 1)))              # no key heads
    norm(view((3, 1, 64), (768, 64, 1)), view((3, 1, 64), (768, 192, 1)))             # one key head
    one = dict(tokens=1, q=view((1, 4, 64), (768, 64, 1)), q_out=view((1, 4, 64), (256, 64, 1)))
    norm(view((1, 2, 64), (768, 64, 1)), view((1, 2, 64), (128, 64, 1)), **one)       # one token
    none = dict(tokens=0, q=empty((0, 4, 64), (768, 64, 1)), q_out=empty((0, 4, 64), (256, 64, 1)))
    norm(empty((0, 2, 64), (768, 64, 1)), empty((0, 2, 64), (128, 64, 1)), **none)
    assert rec.calls == ["qk_norm_rope"] * 4
    for k, k_out in ((view((3, 2, 64), (768, 64, 1)), view((3, 2, 64), (128, 64, 1))),
                     (view((3, 2, 64), (768, 64, 1)), view((3, 2, 64), (768, 128, 1)))):
        with pytest.raises(ValueError, match="strides"):
            norm(k, k_out)
    assert len(rec.calls) == 4


def test_a_step_with_a_bad_output_changes_nothing(cache):
    state = lambda: (cache.lens.tolist(), cache.next_pos.tolist(), list(cache.held))
    before, freq = state(), torch.ones(32)
    qkv = on_gpu(2, 8, 64)

    def at(t, address):
        t.data_ptr = lambda: address
        return t

    far = 2 * FAKE
    for out in (at(on_gpu(2, 4, 128), far), at(on_gpu(1, 4, 64), far), at(on_gpu(2, 256), far), bf16(2, 4, 64),
                at(on_gpu(2, 4, 64, dtype=torch.float32), far), at(on_gpu(1, 4, 64).expand(2, 4, 64), far),
                at(on_gpu(2, 4, 128)[:, :, ::2], far), at(on_gpu(2, 4, 64, gpu=1), far),
                qkv[:, :4], at(qkv[:, 2:6], FAKE + 2 * 128)):
        with pytest.raises(ValueError):
            cache.step(qkv, None, None, freq, out=out)
        assert cache.calls == [] and state() == before
    for out in (at(on_gpu(2, 4, 64), far), at(qkv[:, 4:], FAKE + 4 * 128)):
        assert cache.step(qkv, None, None, freq, out=out) is out
    assert cache.held == [2, 2] and cache.calls == ["sz_qk_norm_rope", "sz_cache_append", "sz_cache_attend"] * 2


def test_a_cache_whose_steps_would_be_refused_is_not_made(S):
    from lossless_kv_cache_bf16_gb300 import decode

    good = dict(batch=2, q_heads=8, kv_heads=4, head_dim=64, max_tokens=64, page_tokens=16, budget=16, recent=4, device="cpu")
    decode.DecodeCache(**good)
    for bad in (dict(q_heads=6), dict(q_heads=0), dict(q_heads=4 * 1025), dict(batch=2049), dict(head_dim=96), dict(kv_heads=0),
                dict(page_tokens=24), dict(budget=0), dict(budget=49), dict(recent=-1)):
        with pytest.raises(ValueError):
            decode.DecodeCache(**{**good, **bad})
