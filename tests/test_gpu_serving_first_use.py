"""The serving operators captured into a CUDA graph on their very first use in
a process (their one-time setup must be legal inside a capture), and called
from several host threads at once on streams of their own."""
import os
import subprocess
import sys

import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, torch
sys.path.insert(0, sys.argv[1])
from lossless_kv_cache_bf16_gb300 import splitzip as S
hq, hk, d, page, b = 8, 2, 128, 16, 3
g = torch.Generator(device="cuda"); g.manual_seed(1)
qkv = torch.randn((b, hq + 2 * hk, d), generator=g, device="cuda").to(torch.bfloat16)
pool = torch.zeros((6, S.sz_cache_page_bytes(d, hk, page)), dtype=torch.uint8, device="cuda")
table = torch.arange(6, dtype=torch.int32, device="cuda").view(b, 2)
slots = table[:, 0].long() * page
lens = torch.ones(b, dtype=torch.int32, device="cuda")
freq = torch.ones(d // 2, device="cuda")
pos = torch.zeros(b, dtype=torch.int32, device="cuda")
weight = torch.zeros((6, hk, page), device="cuda")
where = torch.zeros((6, hk, page), dtype=torch.int32, device="cuda")
q, k = torch.empty((b, hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((b, hk, d), dtype=torch.bfloat16, device="cuda")
out, back, new = torch.empty_like(q), torch.empty_like(k), torch.empty_like(lens)
v = qkv[:, hq + hk:]
ws = torch.empty(S.sz_cache_attend_workspace_size(b, hq, hk, d, 2 * page, True), dtype=torch.uint8, device="cuda")
ews = torch.empty(S.sz_cache_evict_workspace_size(b, hk, 2 * page), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    S.sz_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], None, None, 1e-6, freq, pos, q, k)
    S.sz_cache_append(k, v, slots, pool, page, positions=pos, weight=weight, pos=where)
    S.sz_cache_read(pool, page, slots, k, back)
    S.sz_cache_attend(q, pool, hk, page, table, lens, 0.1, out, ws, weight=weight)
    S.sz_cache_evict(pool, hk, d, page, table, lens, lens, 1, 0, weight, where, new, ews)
graph.replay()
torch.cuda.synchronize()
# One token: the attention is its value, every weight a unit per query head.
want = back.repeat_interleave(hq // hk, dim=1)
assert torch.equal(out, want) and float((back.float() - v.float()).abs().max()) < 0.5
assert torch.allclose(weight[::2, :, 0], torch.full((3, hk), hq / hk, device="cuda"))
assert new.tolist() == [1, 1, 1]
print("ok")
"""


def test_first_use_inside_a_graph_capture():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-4000:]


def test_threads_and_streams():
    import threading

    from lossless_kv_cache_bf16_gb300 import splitzip as S

    hq, hk, d, page, n = 8, 2, 64, 16, 300
    pages = -(-n // page)
    size = S.sz_cache_page_bytes(d, hk, page)
    slots = torch.arange(n, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    inputs, want = [], []
    for i in range(4):
        g = R.gen(i)
        kv = [R.normal_bf16(g, n, hk, d).cuda() for _ in range(2)]
        q = R.normal_bf16(g, 1, hq, d).cuda()
        inputs.append((q, *kv))

    def work(i, stream, results):
        q, k, v = inputs[i]
        with torch.cuda.stream(stream):
            pool = torch.zeros((pages, size), dtype=torch.uint8, device="cuda")
            ws = torch.empty(S.sz_cache_attend_workspace_size(1, hq, hk, d, pages * page), dtype=torch.uint8, device="cuda")
            out = torch.empty_like(q)
            for _ in range(20):
                S.sz_cache_append(k, v, slots, pool, page)
                S.sz_cache_attend(q, pool, hk, page, table, lens, 0.1, out, ws)
            stream.synchronize()
            results[i] = out

    torch.cuda.synchronize()
    alone, together = {}, {}
    for i in range(4):
        work(i, torch.cuda.current_stream(), alone)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, torch.cuda.Stream(), together)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(alone[i], together[i])
