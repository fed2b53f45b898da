"""The host side of the 4-bit cache and of rotated appends: refusals of the C
functions, before any launch, and the reference that the GPU tests use."""
import ctypes

import numpy as np
import pytest

import packed_reference as plain
from test_activation_aware_amd import _capi
from test_serving_host import (ALIGN, BAD_ATTN, BAD_BATCH, INVALID, MIS, NULL, OK, P, SHAPE, UNSUPPORTED, attn, batch, cache,  # noqa: F401
                               lib, ref)

PAGE = 8 * 64 * 80


def packed(**kw):
    d = dict(k=P.value, v=P.value, n_pages=10, page_stride=PAGE, n_kv_heads=8, page_size=64, head_dim=128,
             dtype=_capi.TTQ_F16)
    d.update(kw)
    return _capi.ttq_packed_cache(**d)


def rotation(**kw):
    d = dict(table=P.value, n_positions=100, dim=128, interleaved=0, positions=None)
    d.update(kw)
    return _capi.ttq_rotation(**d)


BAD_PACKED = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=MIS.value), ALIGN), (dict(dtype=_capi.TTQ_F32), UNSUPPORTED),
    (dict(dtype=9), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(n_kv_heads=0), SHAPE), (dict(n_pages=0), SHAPE),
    (dict(page_stride=PAGE - 16), SHAPE), (dict(page_stride=PAGE + 8), ALIGN), (dict(page_stride=1 << 47), SHAPE),
]


def appends(lib, c=None, b=None, r=None, heads=4, q=P, ldq=512, qr=P, ldqr=512, k=P, ldk=1024, v=P, ldv=1024):
    """The status of both appends; they refuse the same calls."""
    r = rotation() if r is None else r
    b = batch() if b is None else b
    rest = (ref(b), None if r == "none" else ref(r), heads, q, ldq, qr, ldqr, k, ldk, v, ldv, None)
    one = lib.ttq_cache_append(ref(cache()), *rest)
    two = lib.ttq_packed_append(ref(packed() if c is None else c), *rest)
    assert c is not None or one == two
    return two


@pytest.mark.parametrize("kw,status", BAD_PACKED)
def test_packed_cache_refusals(lib, kw, status):
    c = packed(**kw)
    assert lib.ttq_packed_append(ref(c), ref(batch()), None, 0, None, 0, None, 0, P, 1024, P, 1024, None) == status
    assert lib.ttq_last_error() != b""
    assert lib.ttq_packed_read(ref(c), ref(batch()), P, 1024, P, 1024, None) == status
    assert lib.ttq_packed_copy_pages(ref(c), 1, 0, P, P, 1, None, 0, 0, 0, None) == status


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_batch_refusals(lib, kw, status):
    assert appends(lib, b=batch(**kw)) == status
    assert lib.ttq_packed_read(ref(packed()), ref(batch(**kw)), P, 1024, P, 1024, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dim=8), SHAPE), (dict(dim=0), SHAPE), (dict(dim=120), SHAPE), (dict(dim=144), SHAPE), (dict(dim=-16), SHAPE),
    (dict(interleaved=2), INVALID), (dict(n_positions=0), SHAPE), (dict(n_positions=1 << 60), SHAPE),
    (dict(table=None), NULL), (dict(table=MIS.value), ALIGN), (dict(positions=MIS.value), ALIGN),
])
def test_rotation_refusals(lib, kw, status):
    assert appends(lib, r=rotation(**kw)) == status


def test_row_refusals(lib):
    assert appends(lib, heads=-1) == SHAPE and appends(lib, heads=16385) == SHAPE
    assert appends(lib, q=None) == NULL and appends(lib, qr=None) == NULL
    assert appends(lib, k=None) == NULL and appends(lib, v=MIS) == ALIGN
    assert appends(lib, ldq=504) == SHAPE and appends(lib, ldqr=516) == ALIGN and appends(lib, ldk=1016) == SHAPE
    assert appends(lib, ldqr=520) == SHAPE          # Q itself, but with another row stride
    assert appends(lib, ldv=1 << 50) == SHAPE
    assert appends(lib, b=batch(total_q=0)) == OK and appends(lib, b=batch(n_seqs=0)) == OK
    assert appends(lib, b=batch(total_q=0x7FFFFFFF), ldq=512) == SHAPE  # more threads than a launch holds
    assert lib.ttq_packed_append(None, ref(batch()), None, 0, None, 0, None, 0, P, 1024, P, 1024, None) == NULL
    assert lib.ttq_packed_read(ref(packed()), ref(batch()), None, 1024, P, 1024, None) == NULL
    assert lib.ttq_packed_read(ref(packed()), ref(batch()), P, 1000, P, 1024, None) == SHAPE
    assert lib.ttq_packed_read(ref(packed()), ref(batch(total_q=1 << 25)), P, 1024, P, 1024, None) == SHAPE


def test_copy_refusals(lib):
    c = packed()

    def copy(layers=1, stride=0, src=P, dst=P, n=1, table=None, rows=0, cols=0, ts=0):
        return lib.ttq_packed_copy_pages(ref(c), layers, stride, src, dst, n, table, rows, cols, ts, None)

    assert copy(layers=0) == SHAPE and copy(layers=2, stride=PAGE - 16) == SHAPE
    assert copy(layers=2, stride=PAGE + 8) == ALIGN and copy(layers=2, stride=1 << 50) == SHAPE
    assert copy(n=-1) == SHAPE and copy(src=None) == NULL and copy(dst=MIS) == ALIGN
    assert copy(table=P, rows=2, cols=4, ts=3) == SHAPE and copy(n=0x7FFFFFFF) == SHAPE
    assert copy(n=0, src=None, dst=None) == OK


def test_a_cache_of_other_bits_is_refused():
    import test_activation_aware_amd as ttq
    with pytest.raises(ValueError):
        ttq.PagedCache(1, 4, 1, 64, bits=8, device="cpu")
    c = ttq.PagedCache(2, 4, 3, 64, page_size=16, bits=4, device="cpu")
    assert c.k.shape == (2, 4, 3, 16, 40)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("keys", [True, False])
def test_the_reference_layout(dim, keys):
    """Every byte of a page has one owner, and what is put is what is got."""
    size = 48
    owners = np.zeros(size * dim * 5 // 8, int)
    for t in range(size):
        words, scales, apart = plain.places(dim, t, keys)
        for w in words:
            assert w % 4 == 0
            owners[w:w + 4] += 1
        for s in scales:
            owners[s:s + 2] += 1
            owners[s + apart:s + apart + 2] += 1
    assert (owners == 1).all()
    rng = np.random.default_rng(0)
    page = rng.integers(0, 256, size * dim * 5 // 8, dtype=np.uint8)
    x = rng.standard_normal((size, dim)).astype(np.float32)
    for t in range(size):
        plain.put(page, t, x[t], keys)
    for t in range(size):
        assert np.array_equal(plain.get(page, t, dim, keys), plain.held(x[t]))
    pages = np.empty((2, 1, size, dim * 5 // 8), np.uint8)
    values = plain.fill(pages, keys, rng)
    assert np.array_equal(plain.get(pages[1, 0].reshape(-1), 17, dim, keys), values[1, 0, 17])


def test_rotation_table():
    import test_activation_aware_amd as ttq
    t = ttq.rotation_table(100, 32, base=500.0, device="cpu").numpy()
    assert t.shape == (100, 32) and t.dtype == np.float32
    assert t[7, 3] == np.float32(np.cos(7 * 500.0 ** (-3 / 16))) and t[99, 16 + 5] == np.float32(np.sin(99 * 500.0 ** (-5 / 16)))


def attend(lib, c=None, b=None, a=None, q=P, ldq=4096, o=P, ldo=4096, lse=None, ws=P, nbytes=1 << 40):
    c, b, a = packed() if c is None else c, batch() if b is None else b, attn() if a is None else a
    return lib.ttq_packed_attention(ref(c), ref(b), ref(a), q, ldq, o, ldo, lse, ws, nbytes, None)


def plan(lib, c=None, b=None, a=None):
    c, b, a = packed() if c is None else c, batch() if b is None else b, attn() if a is None else a
    p = _capi.ttq_packed_plan(9, 9, 9, 9, 9, 9)
    status = lib.ttq_packed_attention_plan(ref(c), ref(b), ref(a), ctypes.byref(p))
    return status, (p.rows, p.waves, p.shares, p.expand_from, p.expand_splits, p.own_table)


@pytest.mark.parametrize("kw,status", BAD_PACKED)
def test_attention_refuses_caches(lib, kw, status):
    c = packed(**kw)
    assert attend(lib, c=c) == status and plan(lib, c=c)[0] == status
    assert lib.ttq_packed_attention_workspace_bytes(ref(c), ref(batch()), ref(attn())) == 0


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_attention_refuses_batches(lib, kw, status):
    b = batch(**kw)
    assert attend(lib, b=b) == status and plan(lib, b=b)[0] == status
    assert lib.ttq_packed_attention_workspace_bytes(ref(packed()), ref(b), ref(attn())) == 0


@pytest.mark.parametrize("kw,status", BAD_ATTN)
def test_attention_refusals(lib, kw, status):
    a = attn(**kw)
    assert attend(lib, a=a) == status and plan(lib, a=a)[0] == status
    assert lib.ttq_packed_attention_workspace_bytes(ref(packed()), ref(batch()), ref(a)) == 0


def test_attention_pointers_and_strides(lib):
    assert attend(lib, q=None) == NULL and attend(lib, o=None) == NULL
    assert attend(lib, q=MIS) == ALIGN and attend(lib, o=MIS) == ALIGN
    assert attend(lib, ldq=4088) == SHAPE and attend(lib, ldo=4100) == ALIGN and attend(lib, ldq=1 << 50) == SHAPE
    assert attend(lib, lse=ctypes.c_void_p((1 << 20) + 1)) == ALIGN
    x = ctypes.POINTER(_capi.ttq_paged_batch)()
    c, b, a = ref(packed()), ref(batch()), ref(attn())
    for args in ((None, b, a), (c, x, a), (c, b, None)):
        assert lib.ttq_packed_attention(*args, P, 4096, P, 4096, None, P, 1 << 40, None) == NULL
        assert lib.ttq_packed_attention_workspace_bytes(*args) == 0
    assert lib.ttq_packed_attention_plan(c, b, a, None) == NULL


def test_attention_of_nothing(lib):
    empty = batch(total_q=0, q_start=None)
    assert attend(lib, b=empty, q=None, o=None, ws=None, nbytes=0) == OK
    assert plan(lib, b=empty) == (OK, (0,) * 6)
    assert attend(lib, b=batch(n_seqs=0)) == SHAPE  # rows of no sequence


@pytest.mark.parametrize("b", [
    dict(n_seqs=2, total_q=2, max_q_len=1, max_kv_len=1 << 16, n_blocks=1 << 10, table_stride=1 << 10),
    dict(n_seqs=3, total_q=2050, max_q_len=2048, max_kv_len=1 << 13, n_blocks=1 << 7, table_stride=1 << 7)])
def test_attention_workspace(lib, b):
    b = batch(**b)
    need = lib.ttq_packed_attention_workspace_bytes(ref(packed()), ref(b), ref(attn()))
    assert need > 0
    assert attend(lib, b=b, nbytes=need - 1) == SHAPE and attend(lib, b=b, nbytes=0) == SHAPE
    assert attend(lib, b=b, ws=None) == NULL and attend(lib, b=b, ws=MIS) == ALIGN


def test_attention_plans(lib):
    """One form for a single sequence, both where prompts may stand beside decode tokens; a
    workspace of pages for the prompts, as many as the batch's blocks or the cache's pages."""
    rows, waves, shares, expand, _, own = plan(lib)[1]
    assert rows in (16, 32) and waves in (1, 4) and shares == 0 and expand == 0
    one = batch(n_seqs=1, total_q=2048, max_q_len=2048, max_kv_len=1 << 13, n_blocks=1 << 7, table_stride=1 << 7)
    rows, _, _, expand, splits, _ = plan(lib, b=one)[1]
    assert rows == 0 and expand == 1 and splits >= 1
    both = batch(n_seqs=3, total_q=2050, max_q_len=2048, max_kv_len=1 << 13, n_blocks=1 << 7, table_stride=1 << 7)
    few, pages = packed(n_pages=100), packed(n_pages=1000)
    assert plan(lib, b=both, c=few)[1][5] == 0 and plan(lib, b=both, c=pages)[1][5] == 1
    assert plan(lib, b=both, c=few)[1][3] > 1 and plan(lib, b=both, c=few)[1][0] > 0
    need = lambda c: lib.ttq_packed_attention_workspace_bytes(ref(c), ref(both), ref(attn()))  # noqa: E731
    page = 2 * 8 * 64 * 128 * 2  # K and V of a page, in 16 bits
    assert need(packed(n_pages=101)) - need(few) == page
    assert need(pages) == need(packed(n_pages=5000)) and need(pages) - need(few) >= (3 * 128 - 100) * page
