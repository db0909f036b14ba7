"""Results that a cache call makes on a stream other than the current one: their memory belongs to that stream."""
import pytest
import torch

from test_gpu_kv_cache import xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream for which the caching allocator holds t's memory."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's memory")


@pytest.mark.parametrize("handle", [False, True])
def test_results_belong_to_the_call_s_stream(xq, handle):  # noqa: F811
    cache = xq.KVCache(8, 8, 16, 2, 64)
    x = torch.randn(128, 2, 64, device="cuda")
    slots = torch.arange(128, device="cuda")
    cache.write(x, x, slots)
    q = torch.randn(1, 1, 4, 64, device="cuda")
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.tensor([128], dtype=torch.int32, device="cuda")
    pre, own, after = table[0, :3].contiguous(), table[:, 3:], lens - 48
    want = cache.attn(q, table, lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    on = s.cuda_stream if handle else s
    out = cache.attn(q, table, lens, stream=on)
    shared = cache.attn_shared(q, pre, 48, own, after, stream=on)
    k, v = cache.read(slots, stream=on)
    s.synchronize()
    for t in (out, shared, k, v):
        assert stream_of(t) == s.cuda_stream
    assert torch.equal(out, want) and k.shape == x.shape
    assert torch.allclose(shared, want, atol=1e-6)
    for t in (want, cache.read(slots)[0]):
        assert stream_of(t) == torch.cuda.current_stream().cuda_stream
