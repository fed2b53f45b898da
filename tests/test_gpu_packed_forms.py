"""Every kernel that attention over the 4-bit cache can take, against 64 bits:
element by element as in test_gpu_packed_attention, with the half step of fp16 for
keys, values and probabilities whatever the type of the rows, and as a whole by the
bound of packed_precision, which roundings to bf16 would break."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import packed_precision as precision  # noqa: E402
from attention_plan import plan as plan16  # noqa: E402
from test_gpu_packed_attention import MODS, PROMPTS, Batch  # noqa: E402

pytestmark = pytest.mark.gpu
SLOPES = [0.5, 0.1, 0.02, 0.0, 0.3, 0.01, 1.0, 0.2]


def check(b, bounds=None, **how):
    got, lse = b.run(bounds, **how)
    want, wl, tol, lse_tol = b.want(u=2.0 ** -11, **how)
    n = len(want)
    assert (got[n:] == 77).all() and (lse[n:] == 77).all()  # rows of no sequence
    bad = np.argwhere(~(np.abs(got[:n] - want) <= tol))
    assert not len(bad), (bad[:5], len(bad))
    again, noise = precision.attend(b, **how)
    assert np.abs(again - want).max() <= 1e-9
    assert precision.off(got[:n], want) <= precision.bound(b.dtype, noise), (precision.off(got[:n], want), noise)
    assert np.array_equal(np.isinf(lse[:n]), np.isinf(wl))
    live = np.isfinite(wl)
    assert (np.abs(lse[:n][live] - wl[live]) <= (lse_tol + 2e-6 * np.abs(wl) + 1e-5)[live]).all()


def kinds(heads):
    """Neither cap nor bias, each, both, and the caps beyond 64: the six kernels of every form."""
    slopes = (SLOPES * heads)[:heads]
    return {"plain": {}, "cap": dict(softcap=20.0), "wide": dict(softcap=100.0), "bias": dict(slopes=slopes),
            "cap+bias": dict(softcap=30.0, slopes=slopes), "wide+bias": dict(softcap=80.0, slopes=slopes)}


KINDS = list(kinds(1))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("longest", [100, 1500])
def test_few_rows(dim, dtype, longest):
    b = Batch([(1, longest), (5, 80), (30, longest), (1, 1), (0, 20)], 8, 2, dim, 16, dtype, spare=1)
    assert b.plan().expand_from == 0
    check(b)
    check(b, window=70)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 10])
def test_one_wave_workgroups(q_len, dim, kind):
    """Contexts of two key tiles at most, and many of them: a wave each, 16 rows of one token or tiles of more."""
    b = Batch([(min(q_len, 1 + i % 40), 1 + i % 40) for i in range(150)], 16, 8, dim, 16,
              "bf16" if (dim // 64 + q_len) % 2 else "f16", spare=2, seed=q_len)
    p = b.plan()
    assert p.waves == 1 and p.shares == 0 and p.expand_from == 0 and p.rows == (16 if q_len == 1 or dim == 256 else 32)
    check(b, **kinds(16)[kind])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("halves", [1, 2])
def test_prompts_of_bf16(halves, dim, kind):
    """fp16 pages under bf16 queries, workgroups of one half and of two, each by the sequences' own lengths."""
    lens = [(140, 140)] * 46 if halves == 1 else [(700, 760), (1, 30), (300, 300), (0, 64)]
    heads, kv_heads = (16, 2) if halves == 1 else (8, 2)
    bounds = (140, 2000) if halves == 1 else (700, 1 << 20)
    b = Batch(lens, heads, kv_heads, dim, 32, "bf16", seed=dim)
    p, rows = b.plan(bounds), max(q for q, _ in lens) * heads // kv_heads
    assert 0 < p.expand_from <= rows
    form, waves, splits = plan16(lens, heads, kv_heads, dim, bounds=bounds)
    assert form == "rows" and waves == 4 * halves and p.expand_splits == splits
    check(b, bounds, **kinds(heads)[kind])


@pytest.mark.parametrize("how", MODS, ids=[",".join(m) + str(i) for i, m in enumerate(MODS)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_masks_of_prompts(dtype, how):
    """Windows and prefixes over a batch whose longest sequence is a prompt by its rows, beside some of few."""
    lens = [(16, 16), (1, 30), (40, 40), (700, 760), (0, 64)]
    b = Batch(lens, 4, 2, 64, 16, dtype)
    if "window" in how:  # with prefixes, though of nothing, a window does not keep the batch from the prompts' way
        how = {"prefix": [0] * 5, **how}
    assert 80 < b.plan(PROMPTS, how.get("window", 0), how.get("prefix")).expand_from <= 1400
    check(b, PROMPTS, **how)
