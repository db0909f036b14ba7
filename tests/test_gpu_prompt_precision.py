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
