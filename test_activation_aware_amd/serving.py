"""Serving operators next to the quantised projections: the paged key-value
cache, attention over it, and token log probabilities.

Functions with the C names (include/ttq.h, "Serving") take torch tensors on
the GPU and enqueue on the current stream of the tensors' device:

    ttq_cache_write       new keys and values into their pages
    ttq_paged_attention   prompt chunks and decode tokens over the cache
    ttq_cache_copy_pages  pages of all layers copied, a block table rewritten
    ttq_token_logprobs    log probabilities, entropy, top alternatives

PagedCache keeps the pages of a model's layers and says which sequence owns
which: it extends, forks, frees and compacts sequences, and hands out the
block table of a batch.  The bookkeeping is on the host, where a scheduler
needs it; the pages move on the GPU.
"""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence

from . import _capi

__all__ = ["PagedCache", "ttq_cache_write", "ttq_paged_attention", "ttq_cache_copy_pages", "ttq_token_logprobs"]

_functions = None


def _torch():
    import torch
    return torch


def _binding():
    """The compiled binding, bound to the loaded library's functions.  Raises
    if either has not been built."""
    global _functions
    if _functions is None:
        _torch()  # its libraries come first
        lib = _capi.load()
        try:
            from . import _binding as binding
        except ImportError as e:
            raise RuntimeError("the serving operators' binding (_binding.so) is missing or does not load: build it "
                               "first (python -m test_activation_aware_amd.build)") from e
        binding.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.ttq_cache_write, lib.ttq_cache_copy_pages, lib.ttq_paged_attention_workspace_bytes,
            lib.ttq_paged_attention, lib.ttq_token_logprobs_workspace_bytes, lib.ttq_token_logprobs)))
        _functions = binding
    return _functions


def ttq_cache_write(K, V, kcache, vcache, block_table, q_start, kv_len) -> None:
    """New keys and values K, V [tokens][kv heads * head dim] (any row stride:
    slices of a fused projection's output will do) into the pages of kcache and
    vcache [pages][kv heads][page size][head dim].

    The tokens are a ragged batch: sequence s owns rows q_start[s] ..
    q_start[s + 1] - 1, its last kv_len[s] positions end with them, and
    position p lies in page block_table[s][p // page size]."""
    status = (_functions or _binding()).cache_write(K, V, kcache, vcache, block_table, q_start, kv_len)
    if status is not None:
        raise _capi.TTQError(status, "ttq_cache_write")


def ttq_paged_attention(Q, kcache, vcache, block_table, q_start, kv_len, max_q_len: int, max_kv_len: int,
                        scale: Optional[float] = None, softcap: float = 0.0, window: int = 0, slopes=None,
                        prefix_len=None, out=None, lse=None, workspace=None):
    """Attention of the new tokens Q [tokens][heads * head dim] over the paged
    cache (with the tokens' own keys and values in it); returns O like Q.

    The batch is described as for ttq_cache_write; max_q_len and max_kv_len
    are its longest lengths, known to the host, or bounds for them (they choose
    among kernels and splits: far from the lengths they cost speed only).
    scale defaults to head dim ** -0.5; softcap > 0 caps the scores by
    softcap * tanh(z / softcap); slopes (fp32 [heads]) subtracts
    slopes[h] * |i - j|; window > 0 limits a query to that many positions up
    to its own; the first prefix_len[s] (int32) positions of a sequence are
    seen by all its queries.  lse (fp32 [tokens][heads]), when given, receives
    the log of the sum of the exponentials.  workspace (uint8) may be passed
    to reuse one buffer; otherwise it is allocated when needed."""
    out = (_functions or _binding()).paged_attention(Q, kcache, vcache, block_table, q_start, kv_len, max_q_len,
                                                     max_kv_len, scale, softcap, window, slopes, prefix_len, out, lse,
                                                     workspace)
    if type(out) is int:
        raise _capi.TTQError(out, "ttq_paged_attention")
    return out


def ttq_cache_copy_pages(kcache, vcache, src, dst, table=None) -> None:
    """Pages src[i] (int32) copied to dst[i] in kcache and vcache, [pages][kv
    heads][page size][head dim] or, for all layers at once, [layers][pages]...;
    with `table` (int32 [rows][blocks]) its entries src[i] become dst[i].  No
    page may be in dst twice, or in both src and dst."""
    status = (_functions or _binding()).cache_copy_pages(kcache, vcache, src, dst, table)
    if status is not None:
        raise _capi.TTQError(status, "ttq_cache_copy_pages")


def ttq_token_logprobs(logits, tokens, top: int = 0, workspace=None):
    """(logprob, entropy) of the tokens (int64 [T]) under logits [T][V] (fp32,
    fp16 or bf16), fp32 [T] each; with top > 0 also the ids (int64 [T][top])
    and log probabilities (fp32) of the most likely alternatives, in order, of
    equal logits the lowest id first.  A token outside [0, V) gets 0."""
    got = (_functions or _binding()).token_logprobs(logits, tokens, top, workspace)
    if type(got) is int:
        raise _capi.TTQError(got, "ttq_token_logprobs")
    return got


class PagedCache:
    """The key-value pages of a model's layers and their owners.

    k, v: [layers][pages][kv heads][page size][head dim] on the GPU.  A
    sequence is named by any hashable value; its pages are counted, so that
    forked sequences share the full ones and copy only the page that both
    would write to.

        cache = PagedCache(layers, pages, kv_heads, head_dim)
        cache.extend("a", 700)                       # room for 700 new tokens
        b = cache.batch(["a"], [700])                # their block table, lengths
        cache.write(layer, K, V, b)
        O = cache.attend(layer, Q, b)
        cache.fork("a", ["b", "c"])                  # decode three answers
        cache.free("b")
        cache.compact()                              # pages in use move to the front
    """

    def __init__(self, layers: int, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, dtype=None,
                 device="cuda"):
        torch = _torch()
        dtype = torch.float16 if dtype is None else dtype
        shape = (layers, pages, kv_heads, page_size, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        self.page_size, self.pages = page_size, pages
        self._free = list(range(pages - 1, -1, -1))  # the lowest page is handed out first
        self._owners = [0] * pages
        self._table: Dict[object, List[int]] = {}
        self._len: Dict[object, int] = {}

    # -- bookkeeping ------------------------------------------------------
    def length(self, seq) -> int:
        return self._len[seq]

    def pages_of(self, seq) -> List[int]:
        return list(self._table[seq])

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def _take(self, n: int) -> List[int]:
        if n > len(self._free):
            raise RuntimeError(f"the cache has {len(self._free)} free pages, {n} are needed")
        got = [self._free.pop() for _ in range(n)]
        for p in got:
            self._owners[p] = 1
        return got

    def _drop(self, page: int) -> None:
        self._owners[page] -= 1
        if self._owners[page] == 0:
            self._free.append(page)

    def extend(self, seq, tokens: int) -> None:
        """Room for `tokens` new positions of seq (new or known).  Its last
        page is its own when it is partly filled (fork copies such a page)."""
        if tokens < 0:
            raise ValueError(f"tokens={tokens} is negative")
        table, length = self._table.get(seq, []), self._len.get(seq, 0)
        self._table[seq] = table + self._take(-(-(length + tokens) // self.page_size) - len(table))
        self._len[seq] = length + tokens

    def fork(self, seq, names: Sequence) -> None:
        """Sequences `names` that continue seq.  They share its full pages and
        get a copy each of the last one when it is partly filled (one launch
        for all of them and all layers)."""
        table, length = self._table[seq], self._len[seq]
        names = list(names)
        if len(set(names)) != len(names) or any(n in self._table for n in names):
            raise ValueError("a forked sequence needs a name of its own")
        part = length % self.page_size != 0
        got = self._take(len(names) if part else 0)
        if got:
            try:
                self._copy([table[-1]] * len(got), got)
            except BaseException:
                for p in reversed(got):
                    self._drop(p)
                raise
        for i, n in enumerate(names):
            shared = table[:-1] if part else list(table)
            for p in shared:
                self._owners[p] += 1
            self._table[n] = shared + ([got[i]] if part else [])
            self._len[n] = length

    def free(self, seq) -> None:
        """Forgets seq; pages that no other sequence shares become free."""
        for p in self._table.pop(seq):
            self._drop(p)
        del self._len[seq]

    def compact(self, table=None) -> int:
        """Moves the pages in use to the front of the cache, so that the rest
        of it is one free piece; returns how many moved.  `table`: a block
        table on the GPU (int32 [rows][blocks]) to be rewritten with them."""
        used = sum(o > 0 for o in self._owners)
        holes = [p for p in range(used) if self._owners[p] == 0]
        moving = [p for p in range(used, self.pages) if self._owners[p] > 0]
        if moving:
            self._copy(moving, holes, table)
            to = dict(zip(moving, holes))
            for a, b in to.items():
                self._owners[b], self._owners[a] = self._owners[a], 0
            for seq, pages in self._table.items():
                self._table[seq] = [to.get(p, p) for p in pages]
        self._free = list(range(self.pages - 1, used - 1, -1))
        return len(moving)

    def _copy(self, src: List[int], dst: List[int], table=None) -> None:
        torch = _torch()
        pairs = torch.tensor([src, dst], dtype=torch.int32).to(self.k.device)
        ttq_cache_copy_pages(self.k, self.v, pairs[0], pairs[1], table)

    # -- the batch of a step ----------------------------------------------
    def batch(self, seqs: Sequence, new_tokens: Sequence[int]) -> dict:
        """What the operators take for a step in which the last new_tokens[i]
        positions of seqs[i] are new: block_table, q_start and kv_len on the
        GPU, and the longest lengths."""
        torch = _torch()
        lens = [self._len[s] for s in seqs]
        if any(n < 0 or n > l for n, l in zip(new_tokens, lens)) or len(new_tokens) != len(lens):
            raise ValueError("new_tokens must be between 0 and each sequence's length")
        blocks = max([len(self._table[s]) for s in seqs] + [1])
        start = [0]
        for n in new_tokens:
            start.append(start[-1] + n)
        flat = start + lens
        for s in seqs:
            flat += self._table[s] + [-1] * (blocks - len(self._table[s]))
        n = len(lens)
        t = torch.tensor(flat, dtype=torch.int32).to(self.k.device)  # one copy for all three
        return {"block_table": t[2 * n + 1:].view(n, blocks), "q_start": t[:n + 1], "kv_len": t[n + 1:2 * n + 1],
                "max_q_len": max(new_tokens, default=0), "max_kv_len": max(lens, default=0)}

    def write(self, layer: int, K, V, batch: dict) -> None:
        ttq_cache_write(K, V, self.k[layer], self.v[layer], batch["block_table"], batch["q_start"], batch["kv_len"])

    def attend(self, layer: int, Q, batch: dict, **how):
        return ttq_paged_attention(Q, self.k[layer], self.v[layer], **batch, **how)
