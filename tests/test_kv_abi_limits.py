"""KV cache entry points: sizes whose products pass 64 bits are refused like other sizes that are too large."""
import ctypes

import pytest

from test_kv_abi import FAKE, cache, query, xq  # noqa: F401 (the fixture)


@pytest.mark.parametrize("kw", [
    dict(batch=1 << 30, n_q=1 << 20, heads=1 << 14),          # 2^64 rows
    dict(batch=(1 << 31) - 1, n_q=1 << 20, heads=1 << 30),
    dict(batch=1 << 30, n_q=1 << 20, heads=(1 << 14) + 2)])
def test_rows_past_64_bits_are_refused(xq, kw):  # noqa: F811
    L, c, q = xq.lib(), cache(xq), query(xq, **kw)
    assert L.xq_kv_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(q)) == 0
    for fn in (L.xq_kv_attn, L.xq_kv_attn_shared):
        assert fn(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 40, None) == 2


def test_the_largest_accepted_sizes(xq):  # noqa: F811
    L, c = xq.lib(), cache(xq)
    for kw in (dict(batch=1 << 28, heads=4), dict(batch=1 << 8, n_q=1 << 20, heads=4), dict(batch=1, heads=1 << 30)):
        assert L.xq_kv_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(query(xq, **kw))) > 0
