"""Prompt attention of 16-bit rows: what the weights' roundings and long sums may add to the result's own rounding."""
import pytest
import torch

import ops_check
from test_gpu_prompt_attn import inputs, starts_of, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,Hk,D,window", [(4, 2, 64, 0), (2, 2, 96, 2), (4, 1, 128, 0), (6, 2, 256, 0), (5, 1, 128, 3)])
def test_what_all_weights_lose_alike_cancels(xq, dtype, H, Hk, D, window):  # noqa: F811
    """Rows of a few keys whose values differ by 2 % around 1 to 2. Weights are divided by their own sum, so their roundings (half
    steps of 2^-8 and 2^-11, as the result's) count with 2 % of their size: 4e-4 of the result's rounding in squares, and fp32's
    sums less. Were they divided by the sum of the weights before rounding, rows of two to nine keys would be off by a further 0.2
    to 0.6 of a rounding. The limit is 1.02."""
    g = torch.Generator("cuda").manual_seed(6)
    starts = starts_of([2 + (5 * i) % 8 for i in range(200)])
    T = starts[-1]
    q, k, v = inputs(T, H, Hk, D, dtype, 7)
    v = (1 + torch.rand(Hk, D, device="cuda", generator=g) + 0.02 * torch.randn(T, Hk, D, device="cuda", generator=g)).to(q.dtype)
    out = xq.prompt_attn(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), window=window)
    want, bound = ops_check.attention(q, k, v, starts, D ** -0.5, window)
    ops_check.within(out, want, bound)
    several = torch.ones(T, dtype=torch.bool, device="cuda")
    several[torch.tensor(starts[:-1])] = False  # a first token sees itself alone: exact
    assert ops_check.rms(out[several], want[several]) <= 1.02 * ops_check.rms(want[several].to(out.dtype), want[several])


@pytest.mark.parametrize("T,D,H,window", [(131071, 128, 8, 0), (60000, 64, 16, 50000), (40000, 256, 4, 0), (40000, 96, 10, 30000)])
def test_long_sums_do_not_drift(xq, T, D, H, window):  # noqa: F811
    """Values of one sign: an addition in a tensor core's accumulator cuts off less than 2^-23 of the sum, always towards 0. A sum
    stays in it for 4096 keys, 256 additions, and grows over them from 0: 2^-23 * 256 / 2 = 1.5e-5 of the result in the mean. The
    mean of results rounded to fp16 at random (half steps of 2^-11 of values of 1 to 2: 2.8e-4 / 1.5) is off by 1.9e-4 / sqrt(1000),
    four times which is 2.4e-5: 3.9e-5 in all."""
    g = torch.Generator("cuda").manual_seed(12)
    q = torch.randn(T, H, D, device="cuda", generator=g).half()
    k = (0.1 * torch.randn(T, H, D, device="cuda", generator=g)).half()
    v = (1 + torch.rand(H, D, device="cuda", generator=g) + 0.05 * torch.randn(T, H, D, device="cuda", generator=g)).half()
    got = xq.prompt_attn(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), window=window)[-1].double()
    first = max(0, T - window) if window else 0
    z = torch.einsum("hd,jhd->hj", q[-1].double(), k[first:].double()) * D ** -0.5
    want = torch.stack([torch.softmax(z[h], -1) @ v[first:, h].double() for h in range(H)])
    assert abs(float(((got - want) / want).mean())) <= 3.9e-5
    assert ops_check.rms(got, want) <= 3e-4  # at random: the result's rounding 2.0e-4, and the weights'
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("slope", [6.0, -6.0, 0.0])
def test_sums_over_runs_of_tiles(xq, dtype, D, slope):  # noqa: F811
    """Keys enough for several runs of tiles whose sums are added up apart; scores that rise (each run has a reference of its
    own), fall (later runs weigh nothing) and neither."""
    lens = [9000, 4097, 4096, 60]
    starts = starts_of(lens)
    T = starts[-1]
    q, k, v = inputs(T, 2, 1, D, dtype, 15)
    if slope:
        at = torch.cat([torch.arange(n, device="cuda") / n for n in lens])
        q[:] = 1.0
        k[:] = (k * 0.02 + slope * at[:, None, None]).to(k.dtype)
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for window in (0, 4500):
        out = xq.prompt_attn(q, k, v, s, scale=64 / D if slope else None, window=window)
        want, bound = ops_check.attention(q, k, v, starts, 64 / D if slope else D ** -0.5, window)
        ops_check.within(out, want, bound)
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_runs_of_tiles_captured_and_side_by_side(xq, dtype):  # noqa: F811
    """Two graphs whose calls have workspaces of their own, replayed at the same time, and a call with a workspace that is handed in."""
    T = 9000
    q, k, v = inputs(T, 4, 2, 128, dtype, 16)
    s = torch.tensor([0, 8900, T], dtype=torch.int32, device="cuda")
    wants = [xq.prompt_attn(q, k, v, s, window=w) for w in (0, 5000)]
    outs, graphs = [], []
    for w in (0, 5000):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(xq.prompt_attn(q, k, v, s, window=w))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], wants[0]) and torch.equal(outs[1], wants[1])
    whole = torch.full((64 << 20,), 7, dtype=torch.uint8, device="cuda")
    xq.prompt_attn(q, k, v, s, out=outs[0], workspace=whole[:32 << 20])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], wants[0]) and bool((whole[32 << 20:] == 7).all())
    with pytest.raises(xq.XQError):
        xq.prompt_attn(q, k, v, s, workspace=whole[:1 << 20])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T", [131071, 524287])
@pytest.mark.parametrize("ahead", [0.1, 0.35, 0.77, 1.3, 2.2, 3.1])
def test_equal_weights_add_up(xq, dtype, T, ahead):  # noqa: F811
    """All keys but the first score alike, so all weights are one number, no power of two, whose additions to a long sum would all be rounded
    one way. Values of 1.5: the result is off by some 3e-5 at most (what the tensor cores cut off), and half a step of it is 3e-4: exact."""
    q = torch.zeros(T, 1, 64, device="cuda", dtype=ops_check.DTYPES[dtype])
    k, v = torch.zeros_like(q), torch.full_like(q, 1.5)
    q[..., 0] = 1
    k[0, 0, 0] = ahead
    out = xq.prompt_attn(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), scale=1.0)
    assert bool((out == 1.5).all())


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 256])
def test_long_rows_by_themselves(xq, dtype, D):  # noqa: F811
    """The last rows see a NaN in one element of V and are computed one by one: equal weights and values of 131071 keys, whose
    additions would all be rounded one way. Sums of 32 terms (2^-24 * 32), then kept exactly: 2^-18 with the quotient, all told.
    At head size 256 fp32 columns 128 and on are computed apart, do not see the NaN, and go the usual way: their sums of outputs and of
    weights are 2048 tiles' each, added in fp32, off by 2^-24 of the running sum, half of the last one in the mean: 2 * 2048 * 2^-25."""
    T = 131071
    q = torch.zeros(T, 1, D, device="cuda", dtype=ops_check.DTYPES[dtype])
    k, v = torch.zeros_like(q), torch.full_like(q, 1.5)
    q[..., 0] = 1
    k[0, 0, 0] = 0.77
    v[T - 20, 0, 9] = float("nan")
    out = xq.prompt_attn(q, k, v, torch.tensor([0, T], dtype=torch.int32, device="cuda"), scale=1.0)[T - 20:, 0]
    assert bool(torch.isnan(out[:, 9]).all())
    out[:, 9] = 1.5
    off = (out.double() / 1.5 - 1).abs()
    alone = 128 if dtype == "fp32" and D == 256 else D
    assert float(off[:, :alone].max()) <= 2.0 ** -18
    assert alone == D or float(off[:, alone:].max()) <= 2.0 ** -18 + 2 * 2048 * 2.0 ** -25
    assert xq.device_error() == 0
