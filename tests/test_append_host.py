"""What PagedCache.append and rotation_table refuse before anything is launched."""
import pytest

import test_activation_aware_amd as ttq
from test_activation_aware_amd import serving

torch = pytest.importorskip("torch")


@pytest.fixture(params=[16, 4])
def cache(request, monkeypatch):
    """A cache on the CPU whose appends are written down."""
    c = ttq.PagedCache(1, 40, 1, 64, page_size=16, bits=request.param, device="cpu")
    c.calls = []
    for name in ("ttq_cache_append", "ttq_packed_append"):
        monkeypatch.setattr(serving, name, lambda *a, _n=name, **kw: c.calls.append((_n, a, kw)))
    return c


def test_positions_past_the_table_are_refused(cache):
    """The kernels would skip such tokens: their keys and values would be missing, without a word."""
    table = ttq.rotation_table(100, 64, device="cpu")
    cache.extend("a", 90)
    cache.extend("b", 30)
    cache.append(0, None, None, None, cache.batch(["a", "b"], [90, 3]), table)
    cache.extend("a", 11)
    for new in ([11, 1], [1, 0], [101, 30]):
        with pytest.raises(ValueError, match="100 positions"):
            cache.append(0, None, None, None, cache.batch(["a", "b"], new), table)
    assert len(cache.calls) == 1


def test_what_needs_no_row_of_the_table(cache):
    table = ttq.rotation_table(100, 64, device="cpu")
    cache.extend("a", 150)
    cache.extend("b", 100)
    b = cache.batch(["a", "b"], [0, 100])            # the long sequence has no new token
    cache.append(0, None, None, None, b, table)
    b = cache.batch(["a"], [20])
    cache.append(0, None, None, None, b, table, positions=torch.zeros(20, dtype=torch.int32))
    cache.append(0, None, None, None, b)             # no rotation
    cache.append(0, None, None, None, b, rotation=None)
    b = cache.batch(["b"], [1])
    cache.append(0, None, None, None, dict(b, max_kv_len=4096), table)  # a bound, as the attention takes it
    assert len(cache.calls) == 5
    assert {n for n, _, _ in cache.calls} == {"ttq_cache_append" if cache.bits == 16 else "ttq_packed_append"}


def test_a_batch_is_what_attention_takes(cache, monkeypatch):
    got = []
    for name in ("ttq_paged_attention", "ttq_packed_attention"):
        monkeypatch.setattr(serving, name, lambda *a, **kw: got.append(kw))
    cache.extend("a", 20)
    cache.attend(0, None, cache.batch(["a"], [2]), window=3)
    assert sorted(got[0]) == ["block_table", "kv_len", "max_kv_len", "max_q_len", "q_start", "window"]


@pytest.mark.parametrize("channels", [1, 33, 63, 0, -2])
def test_rotation_tables_of_odd_channels_are_refused(channels):
    """Pairs are turned: a table of 33 channels would be one of 32 with other angles."""
    with pytest.raises(ValueError):
        ttq.rotation_table(10, channels, device="cpu")
