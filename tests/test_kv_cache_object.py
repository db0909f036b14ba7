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
        held = cache._workspace(key, 0, None)
        assert held[1] >= cache.attn_workspace_bytes(*key)
    assert len(cache._need) <= 1024 and len(cache._ws) == 1
