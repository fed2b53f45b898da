"""Rotated appends where a workgroup has a token's heads in several rounds, and where each round has a workgroup: up to
256 workgroups of them.  A round is 256 threads of 16 channels: 64 heads of 64, 32 of 128, 16 of 256."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_append import Case  # noqa: E402

pytestmark = pytest.mark.gpu
# heads, key heads: the rounds begin inside the queries, the keys or the values, or have queries alone
HEADS = {64: [(100, 20), (70, 35), (128, 4)], 128: [(32, 8), (50, 3), (8, 40)], 256: [(16, 8), (33, 2), (4, 20)]}


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dim,heads,kv_heads", [(d, *h) for d in HEADS for h in HEADS[d]])
def test_rounds_of_heads(dim, heads, kv_heads, packed):
    rounds = -(-(heads + 2 * kv_heads) * dim // 4096)
    assert rounds >= 2
    most = 256 // rounds  # tokens whose rounds have a workgroup each
    for tokens in (most, most + 1):
        lens = ((tokens - 50, tokens), (0, 9), (50, 55))
        Case(dim, heads, kv_heads, 16, "bf16" if dim == 128 else "f16", lens, rotated=dim // 2, packed=packed,
             spare=1 if tokens > most else 0).check(interleaved=dim == 64)
