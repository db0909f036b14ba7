"""Cache attention captured into CUDA graphs without a workspace of the caller's: a graph has memory of its own."""
import gc

import pytest
import torch

from test_gpu_kv_cache import xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def case(xq):  # noqa: F811
    """A cache of 40 pages of 32 tokens, queries of 3 sequences, their table and lengths (cut into parts: the workspace holds
    partial results)."""
    torch.manual_seed(0)
    cache = xq.KVCache(8, 40, 32, 2, 128)
    cache.write(torch.randn(1280, 2, 128, device="cuda"), torch.randn(1280, 2, 128, device="cuda"), torch.arange(1280, device="cuda"))
    table = torch.arange(40, dtype=torch.int32, device="cuda").repeat(3, 1)
    lens = torch.tensor([1280, 700, 1001], dtype=torch.int32, device="cuda")
    return cache, torch.randn(3, 1, 8, 128, device="cuda"), table, lens


def captured(cache, q, table, lens, **kw):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cache.attn(q, table, lens, **kw)
    return g, out


def larger_calls(cache):
    """Calls that need more workspace than the case's, on the streams that it may have used."""
    q = torch.randn(64, 1, 32, 128, device="cuda")
    table = torch.arange(40, dtype=torch.int32, device="cuda").repeat(64, 1)
    lens = torch.full((64,), 900, dtype=torch.int32, device="cuda")
    pre = torch.arange(40, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.current_stream(), torch.cuda.graph.default_capture_stream]
    for s in [x for x in streams if x is not None]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for dtype in (torch.float32, torch.bfloat16):
                cache.attn_shared(q.to(dtype), pre, 1200, table, lens)
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()


def test_a_replay_after_larger_calls(case):
    cache, q, table, lens = case
    g, out = captured(cache, q, table, lens)
    assert not cache._ws  # what a capture takes is not kept for other calls
    want = cache.attn(q, table, lens)
    larger_calls(cache)
    # what the caching allocator has free is taken and filled, as by any other tensor of the program
    others = [torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda") for _ in range(200)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((x == 7).all()) for x in others)


def test_a_graph_outlives_an_earlier_one(case):
    cache, q, table, lens = case
    first, _ = captured(cache, q, table, lens)
    second, out = captured(cache, q, table, lens)
    del first
    gc.collect()
    q.neg_()
    second.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cache.attn(q, table, lens))


def test_two_graphs_beside_each_other(case):
    """Replayed on two streams at a time, in turn: neither uses the other's memory."""
    cache, q, table, lens = case
    other = -2 * q
    a, out_a = captured(cache, q, table, lens)
    b, out_b = captured(cache, other, table, lens)
    want_a, want_b = cache.attn(q, table, lens), cache.attn(other, table, lens)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(50):
        for stream, graph in ((s, a), (t, b)):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_a, want_a) and torch.equal(out_b, want_b)


def test_a_capture_on_a_given_stream(case):
    """The call's stream is captured, not the current one's: the graph's memory is taken all the same."""
    cache, q, table, lens = case
    out = torch.empty_like(q)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        side = torch.cuda.Stream()
        side.wait_stream(s)
        cache.attn(q, table, lens, out=out, stream=side)
        s.wait_stream(side)
    assert not cache._ws
    larger_calls(cache)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cache.attn(q, table, lens))
