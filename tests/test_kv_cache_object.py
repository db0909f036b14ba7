"""KVCache's own checks, without a GPU: pools in host memory, and a current device that is another one."""
import pytest
import torch

from test_kv_abi import xq  # noqa: F401 (the fixture)


@pytest.fixture
def cache(xq):  # noqa: F811
    c = xq.KVCache(8, 4, 16, 2, 64, device="cpu")
    c._device = lambda: 0  # the current device's index; the pools' device is none
    c._current = lambda index: 0
    return c


def test_calls_on_another_device_than_the_current_one_are_refused(cache):
    x, slots = torch.zeros(3, 2, 64), torch.arange(3)
    q, table = torch.zeros(1, 1, 4, 64), torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.ones(1, dtype=torch.int32)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    for call in (lambda: cache.write(x, x, slots), lambda: cache.read(slots),
                 lambda: cache.write(x, x, slots, stream=0), lambda: cache.read(slots, k=x, v=x, stream=0),
                 lambda: cache.attn(q, table, lens), lambda: cache.attn(q, table, lens, workspace=ws),
                 lambda: cache.attn_shared(q, table[0], 20, table, lens, workspace=ws)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_remembered_sizes_are_bounded(cache):
    cache._capturing = lambda: False
    q, lens = torch.float32, 1
    for prefix in range(1, 5000):
        key = (q, 2, 1, 4, lens, prefix)
        held = cache._workspace(key, 0)
        assert held[1] >= cache.attn_workspace_bytes(*key)
    assert len(cache._need) <= 1024 and len(cache._ws) == 1


def test_sizes_past_32_bits_do_not_become_smaller_ones(xq, cache, monkeypatch):  # noqa: F811
    """A window or prefix length reaches the library as it is, as the largest window, or not at all."""
    seen = []

    def entry(ref, query, ws, ws_bytes, stream):
        seen.append((query.window, query.prefix_len))
        return 0
    entry.__name__ = "entry"
    cache._device = lambda: None  # (the pools' device has no index here)
    cache._capturing = lambda: False
    q, table, lens = torch.zeros(1, 1, 4, 64), torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)

    def call(window, prefix_pages=None, prefix_len=0):
        return cache._attn(entry, q, table, lens, None, window, prefix_pages, prefix_len, None, torch.empty(16, dtype=torch.uint8), None)
    for window in (0, 1, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 70):
        call(window)
        assert seen.pop() == (min(window, 2 ** 31 - 1), 0)
    call(-1)
    assert seen.pop() == (-1, 0)  # refused there
    long = torch.zeros(1, dtype=torch.int32).expand(1 << 29)
    monkeypatch.setattr(torch.Tensor, "is_contiguous", lambda self: True)
    for bad in (2 ** 31, 2 ** 32 + 20):
        with pytest.raises(Exception, match="XQ_ERR_SHAPE|2"):
            call(0, long, bad)
    with pytest.raises(Exception):
        call(-2 ** 32 + 5)
    assert not seen
