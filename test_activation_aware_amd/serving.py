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
from ._capi import TTQ_BF16, TTQ_F16, TTQ_F32, check, load

__all__ = ["PagedCache", "ttq_cache_write", "ttq_paged_attention", "ttq_cache_copy_pages", "ttq_token_logprobs"]


def _torch():
    import torch
    return torch


def _stream(t) -> int:
    return _torch().cuda.current_stream(t.device).cuda_stream


def _gpu(t, name: str, dtype, device=None):
    """Checks that t is a GPU tensor of the dtype(s), on `device` when given."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on the GPU{'' if device is None else f' {device}'} (got {t.device})")
    if t.dtype not in dtype if isinstance(dtype, tuple) else t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return t


def _vector(t, name: str, dtype, n: int, device):
    _gpu(t, name, dtype, device)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a dense vector of {n} values (got {tuple(t.shape)})")
    return t.data_ptr()


def _rows(t, name: str, rows: int, cols: int, dtype, device):
    """(pointer, row stride) of a [rows][cols] tensor with unit column stride."""
    _gpu(t, name, dtype, device)
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols or t.stride(1) != 1:
        raise ValueError(f"{name} must be [{rows}][{cols}] with unit column stride (got {tuple(t.shape)}, "
                         f"strides {t.stride()})")
    return t.data_ptr(), t.stride(0) if rows > 1 else max(cols, 8)


def _cache(kcache, vcache):
    """The C description of one layer's cache, k and v [pages][kv heads][page size][head dim]."""
    torch = _torch()
    _gpu(kcache, "kcache", (torch.float16, torch.bfloat16))
    _gpu(vcache, "vcache", kcache.dtype, kcache.device)
    if kcache.dim() != 4 or kcache.shape != vcache.shape:
        raise ValueError("kcache and vcache must be [pages][kv heads][page size][head dim], of one shape "
                         f"(got {tuple(kcache.shape)} and {tuple(vcache.shape)})")
    n, h, p, d = kcache.shape
    stride = kcache.stride(0) if n > 1 else h * p * d
    if (vcache.stride(0) if n > 1 else stride) != stride:
        raise ValueError("kcache and vcache must have one page stride")
    for t in (kcache, vcache):
        if t.stride(3) != 1 or t.stride(2) != d or (h > 1 and t.stride(1) != p * d):
            raise ValueError("a page of the cache must be dense: [kv heads][page size][head dim]")
    return _capi.ttq_paged_cache(kcache.data_ptr(), vcache.data_ptr(), n, stride, h, p, d,
                                 TTQ_F16 if kcache.dtype == torch.float16 else TTQ_BF16)


def _batch(block_table, q_start, kv_len, total_q: int, max_q_len: int, max_kv_len: int, device):
    torch = _torch()
    _gpu(block_table, "block_table", torch.int32, device)
    if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [sequences][blocks] with unit column stride")
    n, blocks = block_table.shape
    return _capi.ttq_paged_batch(_vector(q_start, "q_start", torch.int32, n + 1, device),
                                 _vector(kv_len, "kv_len", torch.int32, n, device), block_table.data_ptr(),
                                 block_table.stride(0) if n > 1 else blocks, blocks, n, total_q, max_q_len, max_kv_len)


def ttq_cache_write(K, V, kcache, vcache, block_table, q_start, kv_len) -> None:
    """New keys and values K, V [tokens][kv heads * head dim] (any row stride:
    slices of a fused projection's output will do) into the pages of kcache and
    vcache [pages][kv heads][page size][head dim].

    The tokens are a ragged batch: sequence s owns rows q_start[s] ..
    q_start[s + 1] - 1, its last kv_len[s] positions end with them, and
    position p lies in page block_table[s][p // page size]."""
    c = _cache(kcache, vcache)
    rows, cols = K.shape[0], c.n_kv_heads * c.head_dim
    k, ldk = _rows(K, "K", rows, cols, kcache.dtype, kcache.device)
    v, ldv = _rows(V, "V", rows, cols, kcache.dtype, kcache.device)
    b = _batch(block_table, q_start, kv_len, rows, 0, 0, kcache.device)
    check(load().ttq_cache_write(ctypes.byref(c), ctypes.byref(b), k, ldk, v, ldv, _stream(kcache)),
          "ttq_cache_write")


def ttq_paged_attention(Q, kcache, vcache, block_table, q_start, kv_len, max_q_len: int, max_kv_len: int,
                        scale: Optional[float] = None, softcap: float = 0.0, window: int = 0, slopes=None,
                        prefix_len=None, out=None, lse=None, workspace=None):
    """Attention of the new tokens Q [tokens][heads * head dim] over the paged
    cache (with the tokens' own keys and values in it); returns O like Q.

    The batch is described as for ttq_cache_write; max_q_len and max_kv_len
    are its longest lengths, known to the host, or bounds for them.  scale
    defaults to head dim ** -0.5; softcap > 0 caps the scores by
    softcap * tanh(z / softcap); slopes (fp32 [heads]) subtracts
    slopes[h] * |i - j|; window > 0 limits a query to that many positions up
    to its own; the first prefix_len[s] (int32) positions of a sequence are
    seen by all its queries.  lse (fp32 [tokens][heads]), when given, receives
    the log of the sum of the exponentials.  workspace (uint8) may be passed
    to reuse one buffer; otherwise it is allocated when needed."""
    torch = _torch()
    c = _cache(kcache, vcache)
    dev = kcache.device
    total, d = Q.shape[0], c.head_dim
    heads = Q.shape[1] // d
    q, ldq = _rows(Q, "Q", total, heads * d, kcache.dtype, dev)
    if out is None:
        out = torch.empty((total, heads * d), dtype=Q.dtype, device=dev)
    o, ldo = _rows(out, "out", total, heads * d, kcache.dtype, dev)
    b = _batch(block_table, q_start, kv_len, total, max_q_len, max_kv_len, dev)
    a = _capi.ttq_attention(heads, d ** -0.5 if scale is None else scale, softcap, window,
                            None if slopes is None else _vector(slopes, "slopes", torch.float32, heads, dev),
                            None if prefix_len is None else
                            _vector(prefix_len, "prefix_len", torch.int32, b.n_seqs, dev))
    if lse is not None:
        _gpu(lse, "lse", torch.float32, dev)
        if lse.shape != (total, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be a dense [{total}][{heads}]")
    lib = load()
    pc, pb, pa = ctypes.byref(c), ctypes.byref(b), ctypes.byref(a)
    need = lib.ttq_paged_attention_workspace_bytes(pc, pb, pa)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        _gpu(workspace, "workspace", torch.uint8, dev)
    check(lib.ttq_paged_attention(pc, pb, pa, q, ldq, o, ldo, None if lse is None else lse.data_ptr(),
                                  None if workspace is None else workspace.data_ptr(),
                                  0 if workspace is None else workspace.numel(), _stream(kcache)),
          "ttq_paged_attention")
    return out


def ttq_cache_copy_pages(kcache, vcache, src, dst, table=None) -> None:
    """Pages src[i] (int32) copied to dst[i] in kcache and vcache, [pages][kv
    heads][page size][head dim] or, for all layers at once, [layers][pages]...;
    with `table` (int32 [rows][blocks]) its entries src[i] become dst[i].  No
    page may be in dst twice, or in both src and dst."""
    torch = _torch()
    layers, stride = 1, 0
    if kcache.dim() == 5:
        layers, stride = kcache.shape[0], kcache.stride(0)
        if vcache.shape != kcache.shape or (layers > 1 and vcache.stride(0) != stride):
            raise ValueError("kcache and vcache must have one shape and one layer stride")
        if layers == 0:
            raise ValueError("a cache of no layers")
        c = _cache(kcache[0], vcache[0])
    else:
        c = _cache(kcache, vcache)
    n = src.shape[0]
    s, t = (_vector(x, name, torch.int32, n, kcache.device) for x, name in ((src, "src"), (dst, "dst")))
    rows = cols = tstride = 0
    tp = None
    if table is not None:
        _gpu(table, "table", torch.int32, kcache.device)
        if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be [rows][blocks] with unit column stride")
        rows, cols = table.shape
        tstride, tp = table.stride(0) if rows > 1 else cols, table.data_ptr()
    check(load().ttq_cache_copy_pages(ctypes.byref(c), layers, stride, s, t, n, tp, rows, cols, tstride,
                                      _stream(kcache)), "ttq_cache_copy_pages")


def ttq_token_logprobs(logits, tokens, top: int = 0, workspace=None):
    """(logprob, entropy) of the tokens (int64 [T]) under logits [T][V] (fp32,
    fp16 or bf16), fp32 [T] each; with top > 0 also the ids (int64 [T][top])
    and log probabilities (fp32) of the most likely alternatives, in order, of
    equal logits the lowest id first.  A token outside [0, V) gets 0."""
    torch = _torch()
    _gpu(logits, "logits", (torch.float32, torch.float16, torch.bfloat16))
    dev = logits.device
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be [T][V] with unit column stride")
    T, V = logits.shape
    tok = _vector(tokens, "tokens", torch.int64, T, dev)
    logprob = torch.empty(T, dtype=torch.float32, device=dev)
    entropy = torch.empty(T, dtype=torch.float32, device=dev)
    ids = lps = None
    if top > 0:
        ids = torch.empty((T, top), dtype=torch.int64, device=dev)
        lps = torch.empty((T, top), dtype=torch.float32, device=dev)
    lib = load()
    need = lib.ttq_token_logprobs_workspace_bytes(T, V, top)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace is not None:
        _gpu(workspace, "workspace", torch.uint8, dev)
    dt = {torch.float32: TTQ_F32, torch.float16: TTQ_F16, torch.bfloat16: TTQ_BF16}[logits.dtype]
    check(lib.ttq_token_logprobs(logits.data_ptr(), dt, T, V, logits.stride(0) if T > 1 else V, tok,
                                 logprob.data_ptr(), entropy.data_ptr(), top, None if ids is None else ids.data_ptr(),
                                 None if lps is None else lps.data_ptr(),
                                 None if workspace is None else workspace.data_ptr(),
                                 0 if workspace is None else workspace.numel(), _stream(logits)),
          "ttq_token_logprobs")
    return (logprob, entropy) if ids is None else (logprob, entropy, ids, lps)


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
            self._copy([table[-1]] * len(got), got)
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
