"""Attention over the 4-bit cache where the cache or the scores are at an end of their range."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import packed_reference as ref  # noqa: E402
from test_gpu_packed_attention import PROMPTS, Batch  # noqa: E402
from test_gpu_packed_forms import check  # noqa: E402

pytestmark = pytest.mark.gpu


# scale and lo: no numbers, or numbers whose codes give none
GARBAGE = ((0x7E00, 0x3C00), (0x7C00, 0x3C00), (0x3C00, 0x7E00), (0x3C00, 0xFC00), (0xFC00, 0xFFFF), (0x7BFF, 0x0000),
           (0xF800, 0x3C00), (0x6C44, 0x7800), (0xEC44, 0xF800), (0x0000, 0x7C00))


def spoil(b, s, position):
    """Garbage for scales and los at a position of sequence s, in both pools and all heads, codes of 0 and 15 among it."""
    page = b.table[s, position // b.page]
    for pool, keys in zip(b.pools, (True, False)):
        words, scales, apart = ref.places(b.dim, position % b.page, keys)
        for h in range(b.kvh):
            flat = pool[page, h].reshape(-1)
            for at in words:
                flat[at:at + 4] = (0xF0, 0xFF, 0x0F, 0x07)
            for i, at in enumerate(scales):
                scale, lo = GARBAGE[(i + h + position) % len(GARBAGE)]
                flat[at:at + 2] = np.array([scale], np.uint16).view(np.uint8)
                flat[at + apart:at + apart + 2] = np.array([lo], np.uint16).view(np.uint8)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len,bounds", [(5, None), (20, None), (90, None), (300, PROMPTS)])
@pytest.mark.parametrize("how", [{}, dict(window=9), dict(window=40, prefix=[3, 0]), dict(softcap=30.0, slopes=[0.5, 0.1, 0.0, 1.0])],
                         ids=["plain", "window", "prefix", "cap"])
def test_positions_that_are_not_seen(how, q_len, bounds, dim, dtype):
    """A position that was skipped over a pool of anything holds scales and los of anything.  A row that does not see it
    (a token before it, or one that it has left the window of) is the same, bit for bit."""
    lens = ((q_len, q_len + 30), (q_len, 2 * q_len))
    b = Batch(lens, 4, 2, dim, 16, dtype)
    if bounds is not None:  # with prefixes, though of nothing, a window does not keep the batch from the prompts' way
        how = {"prefix": [0, 0], **how}
        assert 0 < b.plan(bounds, how.get("window", 0), how["prefix"]).expand_from <= 2 * q_len
    clean, clean_lse = b.run(bounds, **how)
    where = [(0, 30 + q_len // 2), (1, q_len + q_len - 2), (0, 12)]
    for s, p in where:
        spoil(b, s, p)
    dirty, dirty_lse = b.run(bounds, **how)
    unseen = 0
    for s, (ql, kl) in enumerate(lens):
        for t in range(ql):
            at, row = kl - ql + t, b.starts[s] + t
            first = max(0, at - how["window"] + 1) if "window" in how else 0
            if any(q == s and (first <= p <= at or p < how.get("prefix", (0, 0))[s]) for q, p in where):
                continue
            unseen += 1
            assert np.isfinite(dirty[row]).all(), (s, t)
            assert np.array_equal(clean[row], dirty[row]) and np.array_equal(clean_lse[row], dirty_lse[row]), (s, t)
    assert unseen > 0


@pytest.mark.parametrize("bounds", [None, PROMPTS])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("how", [{}, dict(softcap=30.0), dict(slopes=[0.5, 0.01, 0.0, 1.0])], ids=["plain", "cap", "bias"])
def test_the_least_scale(how, dim, dtype, bounds):
    """1e-12, on bf16 queries of 2^-80, below the least power of two that they are divided by: scores of nothing but the
    bias, and rows that see nothing are zeros."""
    b = Batch(((40, 20), (1, 50), (300, 310)), 4, 2, dim, 16, dtype)
    assert (0 < b.plan(bounds).expand_from <= 600) == (bounds is not None)
    if dtype == "bf16":
        b.q = (b.q.float() * 2.0 ** -80).to(b.dtype)
    check(b, bounds, scale=1e-12, **how)
