"""KV cache entry points: sizes and refusals, which return before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from gguf_quant_integer_gb300 import build as xqbuild

FAKE = 1 << 20  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    _xq.lib()
    return _xq


def cache(xq, **kw):
    d = dict(type=8, n_pages=4, page_size=16, heads=2, dim=64, k=FAKE, v=FAKE)
    d.update(kw)
    return xq.xq_kv_cache(**d)


def query(xq, **kw):
    d = dict(type=0, batch=1, n_q=1, heads=4, q=FAKE, out=FAKE, pages=FAKE, page_stride=4, max_pages=4, lens=FAKE, scale=1.0,
             window=0, prefix_pages=FAKE, prefix_len=10)
    d.update(kw)
    return xq.xq_kv_query(**d)


def test_sizes(xq):
    assert xq.kv_bytes(8, 5, 32, 3, 96) == 5 * 32 * 3 * 3 * 34
    assert xq.kv_bytes(2, 5, 32, 3, 96) == 5 * 32 * 3 * 3 * 18
    assert xq.kv_bytes(8, 1 << 20, 64, 8, 128) == (1 << 20) * 64 * 8 * 4 * 34  # past 32 bits
    assert xq.kv_bytes(8, 0, 16, 1, 64) == 0
    for bad in ((12, 1, 16, 1, 64), (8, -1, 16, 1, 64), (8, 1, 24, 1, 64), (8, 1, 8, 1, 64), (8, 1, 8192, 1, 64),
                (8, 1, 16, 0, 64), (8, 1, 16, 1, 32), (8, 1, 16, 1, 100)):
        assert xq.kv_bytes(*bad) == 0
    L = xq.lib()
    ws = lambda c, q: L.xq_kv_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(q))  # noqa: E731
    assert ws(cache(xq), query(xq)) > 0
    assert ws(cache(xq), query(xq, heads=5)) == 0
    assert ws(cache(xq, dim=80), query(xq)) == 0
    assert ws(cache(xq), query(xq, type=8)) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(type=12), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(page_size=48), 2), (dict(dim=32), 2), (dict(heads=0), 2),
    (dict(n_pages=-1), 2), (dict(k=FAKE + 4), 3), (dict(v=FAKE + 8), 3)])
def test_a_bad_cache_is_refused(xq, kw, code):
    L, c, q = xq.lib(), cache(xq, **kw), query(xq)
    assert L.xq_kv_write(ctypes.byref(c), 0, FAKE, 128, FAKE, 128, FAKE, 1, None) == code
    assert L.xq_kv_read(ctypes.byref(c), FAKE, 1, 0, FAKE, FAKE, None) == code
    assert L.xq_kv_attn(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 40, None) == code
    assert L.xq_kv_attn_shared(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 40, None) == code


def test_write_and_read_refusals(xq):
    L, c = xq.lib(), ctypes.byref(cache(xq))
    write = lambda t=0, k=FAKE, ks=128, v=FAKE, vs=128, s=FAKE, n=2: L.xq_kv_write(c, t, k, ks, v, vs, s, n, None)  # noqa: E731
    read = lambda s=FAKE, n=2, t=0, k=FAKE, v=FAKE: L.xq_kv_read(c, s, n, t, k, v, None)  # noqa: E731
    assert L.xq_kv_write(None, 0, FAKE, 128, FAKE, 128, FAKE, 1, None) == 1
    assert write(t=8) == 1 and write(k=None) == 1 and write(v=None) == 1 and write(s=None) == 1
    assert write(n=-1) == 2 and write(ks=127) == 2 and write(vs=0) == 2
    assert write(k=FAKE + 2) == 3 and write(t=1, v=FAKE + 1) == 3 and write(s=FAKE + 4) == 3
    assert write(n=0, k=None, v=None, s=None) == 0
    assert read(t=2) == 1 and read(s=None) == 1 and read(k=None) == 1 and read(v=None) == 1
    assert read(n=-1) == 2 and read(k=FAKE + 4) == 3 and read(v=FAKE + 8) == 3 and read(s=FAKE + 4) == 3
    assert read(n=0, s=None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(type=8), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(pages=None), 1),
    (dict(batch=-1), 2), (dict(n_q=-1), 2), (dict(heads=3), 2), (dict(heads=0), 2), (dict(max_pages=5), 2),
    (dict(max_pages=-1), 2), (dict(window=-1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(max_pages=1 << 27, page_stride=1 << 27), 2), (dict(batch=1 << 30, heads=2048), 2),
    (dict(q=FAKE + 4), 3), (dict(out=FAKE + 8), 3), (dict(pages=FAKE + 2), 3), (dict(lens=FAKE + 1), 3)])
def test_bad_queries_are_refused(xq, kw, code):
    L, c, q = xq.lib(), cache(xq), query(xq, **kw)
    for fn in (L.xq_kv_attn, L.xq_kv_attn_shared):
        assert fn(ctypes.byref(c), ctypes.byref(q), FAKE, 1 << 40, None) == code


def test_shared_refusals_and_empty_calls(xq):
    L, c = xq.lib(), ctypes.byref(cache(xq))
    shared = lambda **kw: L.xq_kv_attn_shared(c, ctypes.byref(query(xq, **kw)), FAKE, 1 << 40, None)  # noqa: E731
    assert shared(prefix_len=-1) == 2 and shared(prefix_pages=None) == 1 and shared(window=5) == 2
    assert shared(prefix_pages=FAKE + 2) == 3
    assert shared(batch=0, q=None) == 0 and shared(n_q=0, q=None) == 0
    assert L.xq_kv_attn(c, None, FAKE, 1 << 40, None) == 1


def test_workspace_is_checked(xq):
    L, c, q = xq.lib(), ctypes.byref(cache(xq)), query(xq)
    assert L.xq_kv_attn(c, ctypes.byref(q), FAKE + 4, 1 << 40, None) == 3
