"""Prompt attention with sequences' bounds out of order: what remains is right, rows that two sequences share apart."""
import pytest
import torch

import ops_check
from test_gpu_prompt_attn import KINDS, inputs, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

# bounds, and how many rows there are
BOUNDS = [([0, 100, 90, 300], 300), ([0, 300, 260, 700, 10, 20], 700), ([50, 0, 200, 150, 400], 420), ([0, 129, 128, 600, 599, 601], 601),
          ([300, 500, 100, 290, 0, 128], 500), ([0, 260, 130, 131, 0, 40], 300), ([5, 5, 5, 4, 5, 64, 0], 64), ([0, 100, 1000, 90, 300], 300)]


def valid(starts, T):
    return [(a, e) for a, e in zip(starts, starts[1:]) if 0 <= a <= e <= T]


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("starts,T", BOUNDS)
@pytest.mark.parametrize("window", [0, 40])
def test_bounds_out_of_order(xq, dtype, D, starts, T, window):  # noqa: F811
    """Every row of one sequence only is that sequence's; rows of none are left as they were; the others are any of theirs, finite."""
    q, k, v = inputs(T, 4, 2, D, dtype, 31)
    # sizes that differ from key tile to key tile, so that each has its own power of two
    size = 2.0 ** (torch.arange(T, device="cuda") * 7 % 5 - 2).float()
    k, v = (k * size[:, None, None]).to(k.dtype), (v * size.flip(0)[:, None, None]).to(v.dtype)
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    assert xq.device_error() == 0
    for _ in range(3):
        out = torch.full_like(q, 7.0)
        xq.prompt_attn(q, k, v, s, window=window, out=out)
        assert xq.device_error() == 5 << 8 | 2
        owners = torch.zeros(T, dtype=torch.int32, device="cuda")
        for a, e in valid(starts, T):
            owners[a:e] += 1
        assert bool((out[owners == 0] == 7.0).all())
        assert bool(torch.isfinite(out[owners > 1]).all())
        for a, e in valid(starts, T):
            if a == e:
                continue
            want, bound = ops_check.attention(q[a:e], k[a:e], v[a:e], [0, e - a], D ** -0.5, window)
            want[owners[a:e] > 1] = float("nan")
            ops_check.within(out[a:e], want, bound, f"{starts} rows {a} to {e}")


def test_bounds_in_order_cost_no_rows_by_themselves(xq):  # noqa: F811
    """Empty sequences, rows of no sequence and bounds past the last token leave the others what they were, bit for bit."""
    q, k, v = inputs(400, 4, 2, 128, "fp32", 32)
    want = xq.prompt_attn(q, k, v, torch.tensor([0, 150, 390], dtype=torch.int32, device="cuda"))
    for starts, error in (([0, 0, 150, 150, 390, 390], 0), ([0, 150, 390, 401], 5 << 8 | 2)):
        got = xq.prompt_attn(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"))
        assert torch.equal(got[:390], want[:390])
        assert xq.device_error() == error
