"""Decoding over a 4-bit paged KV cache, fed by the codec.

The setting of the pages: one machine computes a prompt's KV cache and ships
it as a SplitZip stream, another decodes it bit for bit and generates tokens.
``DecodeCache`` is one layer's cache on that second machine: prompts come in
as bf16 rows or straight from a stream, and every step normalises and rotates
the new query and key, appends K and V, attends, and, with a budget, evicts
the tokens of least accumulated attention weight.  The operators run in the
library's kernels; this module keeps the lengths on the host and on the device,
finds slots (with torch) and calls them in order.  The operators can be captured
in CUDA graphs, a DecodeCache cannot: it decides on the host when to evict.

    python -m lossless_kv_cache_bf16_gb300.decode

runs it on a synthetic prompt and prints what the 4-bit cache and the
eviction change in the attention's result.
"""
from __future__ import annotations

import contextlib
import functools
import math

import torch

from . import splitzip as S


def _on_its_gpu(method):
    """Runs a DecodeCache method with the cache's GPU as the current one, whose
    current stream the library's calls and torch's kernels then share."""
    @functools.wraps(method)
    def call(self, *args, **kwargs):
        with self._gpu():
            return method(self, *args, **kwargs)

    return call


class DecodeCache:
    """One layer's 4-bit cache of `batch` sequences of up to max_tokens tokens.

    budget: tokens a sequence keeps when it has outgrown the budget by a page;
    None keeps every token.  The `recent` last ones are always among them as
    long as recent <= budget, beyond that the budget goes to the weightiest of
    them.  A prompt's tokens come with no weight: what a cut keeps of them goes
    by the steps' queries alone.  A prompt must leave room for a token: a full
    cache refuses steps."""

    def __init__(self, batch: int, q_heads: int, kv_heads: int, head_dim: int, max_tokens: int, page_tokens: int = 64,
                 budget: int | None = None, recent: int = 0, device="cuda"):
        if budget is not None and not 0 < budget <= max_tokens - page_tokens:
            raise ValueError("the budget must leave a page of max_tokens")
        if recent < 0:
            raise ValueError("recent must not be negative")
        self.batch, self.q_heads, self.kv_heads, self.head_dim = batch, q_heads, kv_heads, head_dim
        self.page, self.budget, self.recent = page_tokens, budget, recent
        width = -(-max_tokens // page_tokens)
        pages = batch * width
        size = S.sz_cache_page_bytes(head_dim, kv_heads, page_tokens)
        if size == 0:
            raise ValueError("the cache holds heads of 64 or 128 channels in pages of 16 .. 4,096 tokens, a power of two")
        new = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device=device)
        self.pool = new((pages, size), torch.uint8)
        self.table = torch.arange(pages, dtype=torch.int32, device=device).view(batch, width)
        self.weight = new((pages, kv_heads, page_tokens), torch.float32)
        self.pos = new((pages, kv_heads, page_tokens), torch.int32)
        self.lens, self.spare_lens, self.next_pos = (new(batch, torch.int32) for _ in range(3))
        self.status = new(1, torch.int32)
        self.held = [0] * batch                       # the lengths, as the host knows them
        self.capacity = width * page_tokens
        self.device = self.pool.device
        with self._gpu():
            need = S.sz_cache_attend_workspace_size(batch, q_heads, kv_heads, head_dim, self.capacity, True)
        if need == 0:
            raise ValueError(f"the attention takes up to 2,048 sequences and 1,024 query heads per kv head, not {batch} and "
                             f"{q_heads} over {kv_heads}")
        self.attend_ws = new(need, torch.uint8)
        self.evict_ws = new(S.sz_cache_evict_workspace_size(batch, kv_heads, self.capacity), torch.uint8)

    def _gpu(self):
        return torch.cuda.device(self.device) if self.device.type == "cuda" else contextlib.nullcontext()

    @_on_its_gpu
    def extend(self, sequence: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """Appends a prompt's rows [tokens, kv heads, D], keys already rotated."""
        row = (self.kv_heads, self.head_dim)
        if k.dim() != 3 or k.shape[1:] != row or v.shape != k.shape:
            raise ValueError(f"k and v must be [tokens, {self.kv_heads}, {self.head_dim}], not {tuple(k.shape)} and {tuple(v.shape)}")
        n, at = k.shape[0], self.held[sequence]
        if at + n > self.capacity:
            raise ValueError(f"{at + n} tokens do not fit in {self.capacity}")
        slot = torch.arange(at, at + n, device=self.device)
        slots = self.table[sequence].long()[slot // self.page] * self.page + slot % self.page
        positions = self.next_pos[sequence] + torch.arange(n, dtype=torch.int32, device=self.device)
        S.sz_cache_append(k, v, slots, self.pool, self.page, positions=positions, weight=self.weight, pos=self.pos)
        self.lens[sequence] += n
        self.next_pos[sequence] += n
        self.held[sequence] += n

    @_on_its_gpu
    def extend_from_stream(self, sequence: int, stream: torch.Tensor, nbytes: int, tokens: int) -> None:
        """Appends a prompt that arrives as the SplitZip stream of a bf16
        tensor [2 (K, V), tokens, kv heads, D]."""
        if stream.device != self.device:
            raise ValueError(f"the stream must be on the cache's GPU ({self.device}), not on {stream.device}")
        kv = torch.empty((2, tokens, self.kv_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        S.sz_decode(S.SZ_BF16, stream, nbytes, kv.numel(), kv, self.status)
        self.check()
        self.extend(sequence, kv[0], kv[1])

    def check(self) -> None:
        """Raises if the last call that reported to the status word failed (synchronises)."""
        status = int(self.status.item())
        if status != S.SZ_OK:
            raise S.SplitZipError("DecodeCache", status)

    @_on_its_gpu
    def step(self, qkv: torch.Tensor, q_weight, k_weight, inv_freq: torch.Tensor, eps: float = 1e-6,
             out: torch.Tensor | None = None) -> torch.Tensor:
        """One token of every sequence: qkv [batch, q heads + 2 kv heads, D] as
        a layer's projection gives it, whose queries and keys are normalised and
        rotated in place; returns the attention [batch, q heads, D]."""
        hq, hk = self.q_heads, self.kv_heads
        if qkv.shape != (self.batch, hq + 2 * hk, self.head_dim):
            raise ValueError(f"qkv must be {[self.batch, hq + 2 * hk, self.head_dim]}, not {list(qkv.shape)}")
        if max(self.held) + 1 > self.capacity:
            raise ValueError("the cache is full")
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        shape = (self.batch, hq, self.head_dim)
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        else:  # before the token joins the cache: the attention's own refusal would come after it
            S.check_output(out, shape, q)
        S.sz_qk_norm_rope(q, k, q_weight, k_weight, eps, inv_freq, self.next_pos, q, k)
        at = self.lens.long()
        slots = self.table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page
        S.sz_cache_append(k, v, slots, self.pool, self.page, positions=self.next_pos, weight=self.weight, pos=self.pos)
        self.lens += 1
        self.next_pos += 1
        self.held = [n + 1 for n in self.held]
        S.sz_cache_attend(q, self.pool, hk, self.page, self.table, self.lens, 1 / math.sqrt(self.head_dim), out,
                          self.attend_ws, weight=self.weight, status=self.status)
        if self.budget is not None and max(self.held) >= self.budget + self.page:
            self.evict()
        return out

    @_on_its_gpu
    def evict(self) -> None:
        """Cuts every sequence longer than the budget to it."""
        S.sz_cache_evict(self.pool, self.kv_heads, self.head_dim, self.page, self.table, self.lens, self.next_pos,
                         self.budget, self.recent, self.weight, self.pos, self.spare_lens, self.evict_ws)
        self.lens, self.spare_lens = self.spare_lens, self.lens
        self.held = [min(n, self.budget) for n in self.held]


def _demo(tokens: int = 4096, steps: int = 96, budget: int = 2048) -> None:
    from . import workloads as W

    hq, hk, d = 32, 8, 128
    kv = W.llama8b_prefill("cuda", 0, layers=1, tokens=tokens)[0]
    # The other machine: calibrate, encode.
    n = kv.numel()
    hist = torch.empty(S.sz_histogram_bins(S.SZ_BF16), dtype=torch.int64, device="cuda")
    cb = S.sz_calibrate(S.SZ_BF16, W.llama8b_prefill("cuda", 1, layers=1, tokens=512), hist)
    stream = torch.empty(S.sz_encoded_size(S.SZ_BF16, n, n), dtype=torch.uint8, device="cuda")
    ws = torch.empty(S.sz_workspace_size(S.SZ_BF16, n), dtype=torch.uint8, device="cuda")
    size = torch.zeros(1, dtype=torch.int64, device="cuda")
    S.sz_encode(S.SZ_BF16, cb, kv.contiguous(), stream, size, None, ws)
    nbytes = int(size.item())
    # This machine: two caches of the same prompt, one with a budget.
    full = DecodeCache(1, hq, hk, d, tokens + steps)
    cut = DecodeCache(1, hq, hk, d, tokens + steps, budget=budget, recent=budget // 8)
    for cache in (full, cut):
        cache.extend_from_stream(0, stream, nbytes, tokens)
    print(f"prompt: {tokens} tokens, {2 * n} bytes in bf16, {nbytes} as a stream, {full.lens.item() * hk * (d + d // 8)} in the 4-bit cache")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    freq = 10000.0 ** (-torch.arange(d // 2, device="cuda") * 2.0 / d)
    one = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    for i in range(steps):
        qkv = torch.randn((1, hq + 2 * hk, d), generator=g, device="cuda").to(torch.bfloat16)
        a = full.step(qkv.clone(), one, one, freq)
        b = cut.step(qkv.clone(), one, one, freq)
        if i % 32 == 31:
            off = float((a.float() - b.float()).norm() / a.float().norm())
            print(f"step {i + 1}: {full.held[0]} tokens against {cut.held[0]}, results {off:.3f} apart")
    full.check(), cut.check()


if __name__ == "__main__":
    _demo()
