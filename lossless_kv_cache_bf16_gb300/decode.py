"""Decoding over a 4-bit paged KV cache, fed by the codec.

The setting of the pages: one machine computes a prompt's KV cache and ships
it as a SplitZip stream, another decodes it bit for bit and generates tokens.
``DecodeCache`` is one layer's cache on that second machine: prompts come in
as bf16 rows or straight from a stream, and every step normalises and rotates
the new query and key, appends K and V, attends, and, with a budget, evicts
the tokens of least accumulated attention weight.  A cache without a budget
also takes steps of several drafted tokens: ``draft`` attends for every node of a
tree of them at once, ``accept`` keeps the nodes that a verification
(``sz_verify_tree``) has accepted.  The operators run in the library's kernels; this module keeps the lengths on the host and on the device,
finds slots (with torch) and calls them in order.  The operators can be captured
in CUDA graphs, a DecodeCache cannot: it decides on the host when to evict.

    python -m lossless_kv_cache_bf16_gb300.decode

runs it on a synthetic prompt and prints what the 4-bit cache and the
eviction change in the attention's result, and how many drafted tokens a step
accepts.
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


def tree_masks(parents: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """The trees of parents [batch, nodes] (below a node's own index; any other
    number makes a root) as sz_cache_attend_tree takes them: int64 masks, bit j
    of a node's for itself and each node above it, and every node's int32 depth."""
    nodes = parents.shape[1]
    own = torch.arange(nodes, device=parents.device)
    up = torch.where((parents >= 0) & (parents < own), parents.long(), own)
    depth = (up != own).int()
    mask = (torch.ones_like(own) << own).expand_as(up)
    hops = 1  # of `up`: each turn doubles the part of the way that is known
    while hops < nodes:
        mask, depth, up = mask | mask.gather(1, up), depth + depth.gather(1, up), up.gather(1, up)
        hops *= 2
    return mask.contiguous(), depth


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
        self.drafted = 0                              # nodes that lie behind the lengths
        self.tree_ws = None
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
        self.drafted = 0
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
        self.drafted = 0
        self.lens += 1
        self.next_pos += 1
        self.held = [n + 1 for n in self.held]
        S.sz_cache_attend(q, self.pool, hk, self.page, self.table, self.lens, 1 / math.sqrt(self.head_dim), out,
                          self.attend_ws, weight=self.weight, status=self.status)
        if self.budget is not None and max(self.held) >= self.budget + self.page:
            self.evict()
        return out

    @_on_its_gpu
    def draft(self, qkv: torch.Tensor, parents: torch.Tensor, q_weight, k_weight, inv_freq: torch.Tensor, eps: float = 1e-6,
              counts: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
        """A tree of tokens of every sequence in one pass: qkv [batch, nodes,
        q heads + 2 kv heads, D], node 0 the next token and the others drafted
        behind their parents (int32 [batch, nodes], below a node's own index).
        Queries and keys are normalised and rotated in place, a node's at the
        position that its depth gives it; returns the attention [batch, nodes,
        q heads, D] of every node over the context, the nodes above it and
        itself.  counts (int32 [batch]): nodes of each sequence, if not all; the
        others' results are left as they are, or undefined without out.  With
        them the cache need only have room for the nodes that are there: a full
        sequence takes part with none, and one whose nodes do not fit gets rows
        of zero and is reported by check().  The nodes lie behind the context
        until accept() takes some of them; another draft, step or prompt drops
        them.  No weights are added up, so that a cache with a budget refuses."""
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        if self.budget is not None:
            raise ValueError("a cache with a budget takes no drafts: their steps add up no weights")
        if qkv.dim() != 4 or qkv.shape[0] != self.batch or not 1 <= qkv.shape[1] <= 64 or qkv.shape[2:] != (hq + 2 * hk, d):
            raise ValueError(f"qkv must be [{self.batch}, 1 .. 64, {hq + 2 * hk}, {d}], not {list(qkv.shape)}")
        nodes = qkv.shape[1]
        for name, t, shape in (("parents", parents, (self.batch, nodes)), ("counts", counts, (self.batch,))):
            if t is not None and (t.shape != shape or t.dtype != torch.int32 or t.device != self.device):
                raise ValueError(f"{name} must be int32 of shape {list(shape)} on the cache's GPU")
        over = max(self.held) + nodes > self.capacity
        if over and counts is None:
            raise ValueError("the cache is full")
        shape = (self.batch, nodes, hq, d)
        if out is None:
            out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)
        elif out.shape != shape:
            raise ValueError(f"out must be {list(shape)}, not {list(out.shape)}")
        for name, t in (("qkv", qkv), ("out", out)):
            if self.batch > 1 and nodes > 1 and t.stride(0) != nodes * t.stride(1):
                raise ValueError(f"the sequences of {name} must lie one behind the other")
        rows = qkv.flatten(0, 1)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hk], rows[:, hq + hk:]
        S.check_output(out.flatten(0, 1), (self.batch * nodes, hq, d), q)
        need = S.sz_cache_attend_tree_workspace_size(self.batch, nodes, hq, hk, d, self.capacity)
        if need == 0:
            raise ValueError(f"the attention of trees does not take {nodes} nodes of {self.batch} sequences at this cache's size")
        if self.tree_ws is None or self.tree_ws.numel() < need:
            self.tree_ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        mask, depth = tree_masks(parents)
        positions = (self.next_pos[:, None] + depth).flatten()
        own = torch.arange(nodes, device=self.device)
        at = self.lens.long()[:, None] + own
        if over:  # a node that is not there, or not within the cache, has no slot
            left_out = (at >= self.capacity) | (own >= counts[:, None])
            at = at.clamp_max(self.capacity - 1)
        slots = self.table.gather(1, at // self.page).long() * self.page + at % self.page
        slots = (slots.masked_fill(left_out, -1) if over else slots).flatten()
        S.sz_qk_norm_rope(q, k, q_weight, k_weight, eps, inv_freq, positions, q, k)
        S.sz_cache_append(k, v, slots, self.pool, self.page, positions=positions, weight=self.weight, pos=self.pos)
        self.drafted = nodes
        S.sz_cache_attend_tree(qkv[:, :, :hq], self.pool, hk, self.page, self.table, self.lens, mask, 1 / math.sqrt(d), out,
                               self.tree_ws, counts=counts, status=self.status)
        return out

    @_on_its_gpu
    def accept(self, path: torch.Tensor, accepted: torch.Tensor) -> None:
        """Keeps the nodes of the last draft that path (int32 [batch, nodes])
        names, as many as accepted (int32 [batch]) says, as sz_verify_tree gives
        them, and drops the others.  Waits for the new lengths."""
        if not self.drafted:
            raise ValueError("there is no draft to accept nodes of")
        if path.shape != (self.batch, self.drafted):
            raise ValueError(f"path must be {[self.batch, self.drafted]}, not {list(path.shape)}")
        S.sz_cache_accept(self.pool, self.kv_heads, self.head_dim, self.page, self.table, self.lens, path, accepted,
                          self.spare_lens, weight=self.weight, pos=self.pos, status=self.status)
        self.drafted = 0
        self.next_pos += self.spare_lens - self.lens
        self.lens, self.spare_lens = self.spare_lens, self.lens
        self.held = self.lens.tolist()

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
    _demo_drafts(DecodeCache(1, hq, hk, d, tokens + 256), stream, nbytes, tokens)


def _demo_drafts(cache: DecodeCache, stream: torch.Tensor, nbytes: int, tokens: int, steps: int = 24, vocab: int = 4096) -> None:
    """Generates with a drafter that knows most of the target: the target's
    logits are the drafter's, which go by the last token alone, and a share of
    the attention's."""
    hq, hk, d = cache.q_heads, cache.kv_heads, cache.head_dim
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    embed = normal(vocab, hq + 2 * hk, d).to(torch.bfloat16)
    likely, head = 4 * normal(vocab, vocab), (normal(hq * d, vocab) / math.sqrt(d)).to(torch.bfloat16)
    freq = 10000.0 ** (-torch.arange(d // 2, device="cuda") * 2.0 / d)
    one = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    # A node with three children, of which each has one more, and so on.
    parents = torch.tensor([[0, 0, 0, 0, 1, 2, 3, 4, 5, 6]], dtype=torch.int32, device="cuda")
    nodes = parents.shape[1]
    path, accepted, token = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, nodes), (1,), (1,)))
    cache.extend_from_stream(0, stream, nbytes, tokens)
    for _ in range(steps):
        drafted = token.expand(nodes).clone()
        drafted[1:4] = likely[token[0]].topk(3).indices
        for j in range(4, nodes):
            drafted[j] = likely[drafted[parents[0, j]]].argmax()
        out = cache.draft(embed[drafted][None], parents, one, one, freq)
        logits = likely[drafted] + (out[0].flatten(1) @ head).float()
        S.sz_verify_tree(logits[None], drafted[None], parents, 1.0, path, accepted, token,
                         uniforms=torch.rand((1, nodes), generator=g, device="cuda"),
                         noise=torch.empty((1, vocab), device="cuda").exponential_(generator=g), status=cache.status)
        cache.check()
        cache.accept(path, accepted)
    cache.check()
    print(f"drafts of {nodes - 1}: {steps} steps added {cache.held[0] - tokens} tokens")


if __name__ == "__main__":
    _demo()
