"""The host side of the 4-bit cache and of rotated appends: refusals of the C
functions, before any launch, and the reference that the GPU tests use."""
import ctypes

import numpy as np
import pytest

import packed_reference as plain
from test_activation_aware_amd import _capi
from test_serving_host import ALIGN, BAD_BATCH, INVALID, MIS, NULL, OK, P, SHAPE, UNSUPPORTED, batch, cache, lib, ref  # noqa: F401

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
