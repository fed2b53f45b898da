"""The least scale of attention over the 4-bit cache."""
import pytest

from test_packed_host import attend, packed, plan
from test_serving_host import INVALID, OK, attn, batch, cache, lib, ref  # noqa: F401


@pytest.mark.parametrize("scale", [1e-13, 1e-30, 1e-45])
def test_scales_below_the_least_are_refused(lib, scale):
    """With bf16 queries near 0 they would be nothing in 32 bits, and rows that see nothing NaN."""
    a = attn(scale=scale)
    assert attend(lib, a=a) == INVALID and b"scale" in lib.ttq_last_error()
    assert plan(lib, a=a)[0] == INVALID
    b = batch(total_q=2, max_kv_len=1 << 16, n_blocks=1 << 10, table_stride=1 << 10)
    assert lib.ttq_packed_attention_workspace_bytes(ref(packed()), ref(b), ref(a)) == 0


def test_the_least_scale_is_taken(lib):
    a = attn(scale=1e-12)
    assert plan(lib, a=a)[0] == OK
    b = batch(total_q=2, max_kv_len=1 << 16, n_blocks=1 << 10, table_stride=1 << 10)
    assert lib.ttq_packed_attention_workspace_bytes(ref(packed()), ref(b), ref(a)) > 0
    assert lib.ttq_paged_attention_workspace_bytes(ref(cache()), ref(b), ref(attn(scale=1e-30))) > 0
