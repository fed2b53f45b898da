"""The serving operators' host side: what they refuse, the workspaces they ask
for, and the page bookkeeping of PagedCache.  Nothing here reaches a launch."""
import ctypes

import pytest

from test_activation_aware_amd import _capi

P = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 2)
OK, INVALID, UNSUPPORTED, SHAPE, NULL, ALIGN = (_capi.TTQ_OK, _capi.TTQ_ERR_INVALID_ARG, _capi.TTQ_ERR_UNSUPPORTED,
                                                _capi.TTQ_ERR_SHAPE, _capi.TTQ_ERR_NULL, _capi.TTQ_ERR_ALIGN)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_capi.LIB_PATH):
        from test_activation_aware_amd.build import build
        build()
    return _capi.load()


def cache(**kw):
    d = dict(k=P.value, v=P.value, n_pages=10, page_stride=8 * 64 * 128, n_kv_heads=8, page_size=64, head_dim=128,
             dtype=_capi.TTQ_F16)
    d.update(kw)
    return _capi.ttq_paged_cache(**d)


def batch(**kw):
    d = dict(q_start=P.value, kv_len=P.value, block_table=P.value, table_stride=4, n_blocks=4, n_seqs=2, total_q=2,
             max_q_len=1, max_kv_len=200)
    d.update(kw)
    return _capi.ttq_paged_batch(**d)


def attn(**kw):
    d = dict(n_heads=32, scale=0.1, softcap=0.0, window=0, slopes=None, prefix_len=None)
    d.update(kw)
    return _capi.ttq_attention(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHE = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS.value), ALIGN), (dict(dtype=_capi.TTQ_F32), UNSUPPORTED),
    (dict(dtype=7), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), SHAPE),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=-1), SHAPE),
    (dict(n_kv_heads=0), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE),
    (dict(page_stride=8 * 64 * 128 - 8), SHAPE), (dict(page_stride=8 * 64 * 128 + 4), ALIGN),
    (dict(page_stride=1 << 47), SHAPE),
]
BAD_BATCH = [
    (dict(n_seqs=-1), SHAPE), (dict(total_q=-1), SHAPE), (dict(total_q=1 << 31), SHAPE), (dict(max_q_len=-1), SHAPE),
    (dict(max_kv_len=-5), SHAPE), (dict(n_blocks=0), SHAPE), (dict(table_stride=3), SHAPE),
    (dict(table_stride=1 << 60), SHAPE), (dict(q_start=None), NULL), (dict(kv_len=None), NULL),
    (dict(block_table=None), NULL), (dict(block_table=MIS.value), ALIGN),
]
BAD_ATTN = [
    (dict(n_heads=12), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_heads=1 << 20), SHAPE), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID), (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(slopes=MIS.value), ALIGN),
    (dict(prefix_len=MIS.value), ALIGN),
]


def call_attention(lib, c, b, a, q=P, ldq=4096, o=P, ldo=4096, lse=None, ws=P, nbytes=1 << 40):
    return lib.ttq_paged_attention(ref(c), ref(b), ref(a), q, ldq, o, ldo, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_refusals(lib, kw, status):
    c, b = cache(**kw), batch()
    assert lib.ttq_cache_write(ref(c), ref(b), P, 1024, P, 1024, None) == status, lib.ttq_last_error()
    assert lib.ttq_last_error() != b""
    assert call_attention(lib, c, b, attn()) == status
    assert lib.ttq_cache_copy_pages(ref(c), 1, 0, P, P, 1, None, 0, 0, 0, None) == status
    assert lib.ttq_paged_attention_workspace_bytes(ref(c), ref(b), ref(attn())) == 0


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batch_refusals(lib, kw, status):
    c, b = cache(), batch(**kw)
    assert lib.ttq_cache_write(ref(c), ref(b), P, 1024, P, 1024, None) == status, lib.ttq_last_error()
    assert call_attention(lib, c, b, attn()) == status


@pytest.mark.parametrize("kw,status", BAD_ATTN)
def test_attention_refusals(lib, kw, status):
    assert call_attention(lib, cache(), batch(), attn(**kw)) == status, lib.ttq_last_error()


def test_tensor_refusals(lib):
    c, b, a = cache(), batch(), attn()
    assert call_attention(lib, c, b, a, q=None) == NULL
    assert call_attention(lib, c, b, a, o=None) == NULL
    assert call_attention(lib, c, b, a, q=MIS) == ALIGN
    assert call_attention(lib, c, b, a, ldq=4088) == SHAPE
    assert call_attention(lib, c, b, a, ldo=4100) == ALIGN
    assert call_attention(lib, c, b, a, ldq=1 << 50) == SHAPE
    assert call_attention(lib, c, b, a, lse=ctypes.c_void_p((1 << 20) + 1)) == ALIGN
    for x in (None,):
        assert call_attention(lib, x, b, a) == NULL
        assert call_attention(lib, c, x, a) == NULL
        assert call_attention(lib, c, b, x) == NULL
    assert call_attention(lib, c, batch(n_seqs=0), a) == SHAPE         # rows of no sequence
    assert call_attention(lib, c, batch(total_q=0, q_start=None), a, q=None, o=None) == OK  # nothing to do
    big = batch(total_q=0x7FFFFFFF // 32 + 1)
    assert call_attention(lib, c, big, a) == SHAPE
    # write: K too narrow, V misaligned, nothing to do
    assert lib.ttq_cache_write(ref(c), ref(b), P, 1016, P, 1024, None) == SHAPE
    assert lib.ttq_cache_write(ref(c), ref(b), P, 1024, MIS, 1024, None) == ALIGN
    assert lib.ttq_cache_write(ref(c), ref(b), None, 1024, P, 1024, None) == NULL
    assert lib.ttq_cache_write(ref(c), ref(batch(n_seqs=0, total_q=0)), None, 0, None, 0, None) == OK


def test_copy_refusals(lib):
    c = cache()

    def copy(layers=1, stride=0, src=P, dst=P, n=1, table=None, rows=0, cols=0, ts=0):
        return lib.ttq_cache_copy_pages(ref(c), layers, stride, src, dst, n, table, rows, cols, ts, None)

    assert copy(layers=0) == SHAPE and copy(layers=1 << 20) == SHAPE
    assert copy(layers=2, stride=64) == SHAPE and copy(layers=2, stride=(1 << 20) + 4) == ALIGN
    assert copy(layers=2, stride=1 << 50) == SHAPE
    assert copy(n=-1) == SHAPE and copy(src=None) == NULL and copy(dst=MIS) == ALIGN
    assert copy(table=P, rows=2, cols=4, ts=3) == SHAPE and copy(table=P, rows=-1, cols=1, ts=1) == SHAPE
    assert copy(table=MIS, rows=2, cols=4, ts=4) == ALIGN
    assert copy(n=0x7FFFFFFF) == SHAPE                                  # too many for one launch
    assert copy(n=0, src=None, dst=None) == OK


def test_logprobs_refusals(lib):
    def f(x=P, dt=0, T=4, V=100, ldl=100, tok=P, lp=P, en=P, top=5, ids=P, tl=P, ws=P, n=1 << 40):
        return lib.ttq_token_logprobs(x, dt, T, V, ldl, tok, lp, en, top, ids, tl, ws, n, None)

    assert f(dt=7) == INVALID and f(T=-1) == SHAPE and f(V=0, ldl=0) == SHAPE and f(V=(1 << 23) + 1, ldl=1 << 24) == SHAPE
    assert f(ldl=99) == SHAPE and f(ldl=1 << 50) == SHAPE and f(top=-1) == INVALID and f(top=65) == INVALID
    assert f(V=4, ldl=4) == SHAPE                                       # top > V
    assert f(x=None) == NULL and f(x=MIS) == ALIGN and f(dt=1, x=ctypes.c_void_p((1 << 20) + 1)) == ALIGN
    assert f(tok=None) == NULL and f(tok=ctypes.c_void_p((1 << 20) + 4)) == ALIGN
    assert f(lp=None) == NULL and f(en=MIS) == ALIGN and f(ids=None) == NULL and f(tl=None) == NULL
    need = lib.ttq_token_logprobs_workspace_bytes(1, 100000, 5)
    assert need > 0
    assert f(T=1, V=100000, ldl=100000, n=need - 1) == SHAPE and f(T=1, V=100000, ldl=100000, ws=None) == NULL
    assert f(T=0, x=None, tok=None) == OK
    assert lib.ttq_token_logprobs_workspace_bytes(4, 100, 65) == 0
    assert lib.ttq_token_logprobs_workspace_bytes(100000, 100000, 5) == 0   # whole rows


def test_attention_workspace(lib):
    # one decode token over a long context is split: fp32 partial outputs, maxima and sums
    c, b, a = cache(), batch(n_seqs=1, total_q=1, max_kv_len=1 << 17, n_blocks=2048, table_stride=2048), attn()
    need = lib.ttq_paged_attention_workspace_bytes(ref(c), ref(b), ref(a))
    assert need > 0 and (need - 32 * 4) % (32 * (128 * 4 + 8)) == 0
    assert call_attention(lib, c, b, a, nbytes=need - 1) == SHAPE
    assert call_attention(lib, c, b, a, ws=None) == NULL
    # enough rows: none
    full = batch(n_seqs=1, total_q=1 << 16, max_q_len=1 << 16, max_kv_len=1 << 16, n_blocks=1024, table_stride=1024)
    assert lib.ttq_paged_attention_workspace_bytes(ref(c), ref(full), ref(a)) == 0


# -- PagedCache ------------------------------------------------------------
@pytest.fixture
def paged():
    pytest.importorskip("torch")
    from test_activation_aware_amd import PagedCache

    class Recorded(PagedCache):  # the bookkeeping alone: what would move is written down
        def _copy(self, src, dst, table=None):
            self.moves = getattr(self, "moves", []) + list(zip(src, dst))

    return Recorded(2, 12, 1, 64, page_size=16, device="cpu")


def check_owners(c):
    owned = {}
    for s, pages in c._table.items():
        assert len(pages) == -(-c.length(s) // c.page_size)
        for p in pages:
            owned[p] = owned.get(p, 0) + 1
    assert [owned.get(p, 0) for p in range(c.pages)] == c._owners
    assert sorted(c._free) == [p for p in range(c.pages) if p not in owned]


def test_paged_cache_extend_fork_free(paged):
    paged.extend("a", 40)
    assert paged.pages_of("a") == [0, 1, 2] and paged.length("a") == 40
    paged.extend("a", 8)                       # fills the third page
    assert paged.pages_of("a") == [0, 1, 2]
    paged.extend("a", 1)
    assert paged.pages_of("a") == [0, 1, 2, 3]
    check_owners(paged)
    paged.fork("a", ["b", "c"])                # the last page is partly filled: a copy for each
    assert paged.moves == [(3, 4), (3, 5)] and paged.pages_of("b") == [0, 1, 2, 4]
    check_owners(paged)
    paged.extend("b", 16)
    assert paged.pages_of("b") == [0, 1, 2, 4, 6]
    paged.free("a")
    assert paged.free_pages == 12 - 6 and paged.pages_of("c") == [0, 1, 2, 5]
    check_owners(paged)
    paged.extend("d", 32)
    paged.fork("d", ["e"])                     # full pages only: nothing to copy
    assert len(paged.moves) == 2 and paged.pages_of("d") == paged.pages_of("e")
    paged.extend("d", 1)
    assert paged.pages_of("d")[:2] == paged.pages_of("e")
    check_owners(paged)
    for s in "bcde":
        paged.free(s)
    assert paged.free_pages == 12
    check_owners(paged)


def test_paged_cache_compact(paged):
    for s in "abcd":
        paged.extend(s, 40)
    paged.free("a")
    paged.free("c")
    was = {s: paged.pages_of(s) for s in "bd"}
    assert paged.compact() == 3
    assert all(a not in [d for _, d in paged.moves] for a, _ in paged.moves)
    to = dict(paged.moves)
    assert all(d < 6 <= s for s, d in paged.moves)
    assert {s: paged.pages_of(s) for s in "bd"} == {s: [to.get(p, p) for p in was[s]] for s in "bd"}
    check_owners(paged)
    assert paged.compact() == 0
    paged.extend("e", 16)
    assert paged.pages_of("e") == [6]


def test_paged_cache_refusals(paged):
    paged.extend("a", 100)
    with pytest.raises(RuntimeError, match="free pages"):
        paged.extend("b", 100)
    check_owners(paged)                        # nothing was taken
    with pytest.raises(RuntimeError, match="free pages"):
        paged.fork("a", list("bcdefg"))
    with pytest.raises(ValueError):
        paged.fork("a", ["a"])
    with pytest.raises(ValueError):
        paged.extend("a", -1)
    with pytest.raises(ValueError):
        paged.batch(["a"], [101])
    with pytest.raises(KeyError):
        paged.free("z")
    check_owners(paged)


def test_paged_cache_batch(paged):
    paged.extend("a", 20)
    paged.extend("b", 5)
    paged.extend("c", 0)
    b = paged.batch(["b", "a", "c"], [5, 1, 0])
    assert b["block_table"].tolist() == [[2, -1], [0, 1], [-1, -1]]
    assert b["q_start"].tolist() == [0, 5, 6, 6] and b["kv_len"].tolist() == [5, 20, 0]
    assert b["max_q_len"] == 5 and b["max_kv_len"] == 20


# -- the Python functions: what they refuse before the library is called -----
def test_binding_refuses_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    import test_activation_aware_amd as ttq
    x = torch.zeros((2, 64), dtype=torch.float16)
    c = torch.zeros((4, 1, 16, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="kcache must be on the GPU"):
        ttq.ttq_paged_attention(x, c, c, i[None], i, i[:1], 1, 1)
    with pytest.raises(ValueError, match="on the GPU"):
        ttq.ttq_cache_write(x, x, c, c, i[None], i, i[:1])
    with pytest.raises(ValueError, match="on the GPU"):
        ttq.ttq_cache_copy_pages(c, c, i, i)
    with pytest.raises(ValueError, match="logits must be on the GPU"):
        ttq.ttq_token_logprobs(x, i)
    with pytest.raises(TypeError, match="logits must be a torch tensor"):
        ttq.ttq_token_logprobs([1.0], i)


# -- the plan of an attention call ---------------------------------------------
def test_attention_plan(lib):
    """One form a call, by its sizes: what the forms' own tests and documents say of them."""
    from attention_plan import plan
    assert plan([(1, 333)], 12, 12, 64) == ("keys", 4, 1)
    assert plan([(1, 500)] * 128, 32, 8, 128) == ("keys", 1, 1)
    assert plan([(1, 131072)] * 3, 32, 8, 128)[:2] == ("keys", 4)
    assert plan([(1, 131072)] * 3, 32, 8, 128)[2] > 2
    assert plan([(1, 5000)], 8, 1, 256)[:2] == ("keys", 2)
    assert plan([(4096, 10000)], 64, 8, 128) == ("rows", 4, 1)
    assert plan([(1000, 3000)], 32, 8, 128) == ("rows", 8, 1)
    form = plan([(64, 16000)], 32, 8, 128)
    assert form[:2] == ("rows", 8) and form[2] > 2
    p = _capi.ttq_attention_plan(form=9, waves=9, splits=9)
    call = lambda c, b, a, to: lib.ttq_paged_attention_plan(ref(c), ref(b), ref(a), to)  # noqa: E731
    assert call(cache(), batch(total_q=0), attn(), ctypes.byref(p)) == OK and (p.form, p.waves, p.splits) == (0, 0, 0)
    assert call(cache(), batch(), attn(), None) == NULL
    assert call(cache(head_dim=96), batch(), attn(), ctypes.byref(p)) == UNSUPPORTED
    assert call(cache(), batch(n_seqs=-1), attn(), ctypes.byref(p)) == SHAPE
    assert call(cache(), batch(), attn(scale=0.0), ctypes.byref(p)) == INVALID


def test_paged_cache_keeps_its_books_when_a_copy_fails(paged):
    """fork and compact whose copy raises: pages, owners and names as before."""
    for s in "abc":
        paged.extend(s, 20)
    paged.free("a")
    before = (list(paged._free), list(paged._owners), {s: paged.pages_of(s) for s in "bc"})

    def fails(src, dst, table=None):
        raise RuntimeError("no launch")

    works, paged._copy = paged._copy, fails
    with pytest.raises(RuntimeError, match="no launch"):
        paged.fork("b", ["d", "e"])
    with pytest.raises(RuntimeError, match="no launch"):
        paged.compact()
    assert sorted(paged._free) == sorted(before[0])
    assert (paged._owners, {s: paged.pages_of(s) for s in "bc"}) == before[1:]
    check_owners(paged)
    paged._copy = works
    paged.fork("b", ["d", "e"])
    check_owners(paged)


def test_sizes_beyond_one_launch_are_refused(lib):
    """A launch holds less than 2^32 threads; larger calls are named as such and not tried."""
    c = cache()
    n = 1 << 20                                          # pairs of 16 pieces each, keys and values: 2^33 threads
    assert lib.ttq_cache_copy_pages(ref(c), 1, 0, P, P, n, None, 0, 0, 0, None) == SHAPE
    assert b"one launch" in lib.ttq_last_error()
    rows = 1 << 28                                       # four a workgroup of 256
    assert lib.ttq_cache_write(ref(c), ref(batch(total_q=rows)), P, 1024, P, 1024, None) == SHAPE
    assert b"one launch" in lib.ttq_last_error()
    b = batch(n_seqs=1 << 24, total_q=1 << 24)           # a workgroup or more for each sequence and key head
    assert call_attention(lib, c, b, attn(), nbytes=1 << 50) == SHAPE
    assert b"one launch" in lib.ttq_last_error()
    assert lib.ttq_token_logprobs(P, 1, 1 << 27, 10, 10, P, P, P, 0, None, None, None, 0, None) == SHAPE
    assert b"one launch" in lib.ttq_last_error()
