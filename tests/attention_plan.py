"""The plan of an attention call, asked of the library on the host: which form a
test's sizes run in."""
import ctypes

from test_activation_aware_amd import _capi

FORMS = {_capi.TTQ_ATTENTION_KEYS: "keys", _capi.TTQ_ATTENTION_ROWS: "rows"}


def plan(lens, heads, kv_heads, dim, window=0, prefix=None, bounds=None, **_):
    """(form, waves of a workgroup, splits) for sequences of (new tokens, keys)."""
    some = ctypes.c_void_p(1 << 20)  # described, not touched
    max_q, max_kv = bounds or (max(q for q, _ in lens), max(k for _, k in lens))
    c = _capi.ttq_paged_cache(k=some.value, v=some.value, n_pages=1, page_stride=kv_heads * 16 * dim,
                              n_kv_heads=kv_heads, page_size=16, head_dim=dim, dtype=_capi.TTQ_F16)
    b = _capi.ttq_paged_batch(q_start=some.value, kv_len=some.value, block_table=some.value, table_stride=1, n_blocks=1,
                              n_seqs=len(lens), total_q=sum(q for q, _ in lens), max_q_len=max_q, max_kv_len=max_kv)
    a = _capi.ttq_attention(n_heads=heads, scale=1.0, softcap=0.0, window=window, slopes=None,
                            prefix_len=None if prefix is None else some.value)
    p = _capi.ttq_attention_plan()
    status = _capi.load().ttq_paged_attention_plan(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), ctypes.byref(p))
    _capi.check(status, "ttq_paged_attention_plan")
    return FORMS[p.form], p.waves, p.splits
