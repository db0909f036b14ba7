"""Prompt attention's waits: one that runs out is recorded and leaves the context usable, and none does behind slow work.

A test hook (xq_debug_stalled_prompt_attn) cuts the waits' limit to a short time beside what slow work is allowed, by itself or with
the copies withheld. No GPU fault is involved: a wait that runs out ends the kernel's loops."""
import math

import pytest
import torch

import ops_check
from test_gpu_prompt_attn import KINDS, inputs, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

SHORT = 400_000  # clocks, 0.2 ms: some fifty times what an item's copies take


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_withheld_copies_are_reported(xq, dtype, D):  # noqa: F811
    assert xq.device_error() == 0
    q, k, v = inputs(700, 4, 2, D, dtype, 41)
    s = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    xq.debug_stalled_prompt_attn(q, k, v, s, SHORT, True, out=out)
    assert xq.device_error() >> 8 == 6
    assert bool((out == 7.0).all())
    assert xq.device_error() == 0
    xq.prompt_attn(q, k, v, s, out=out)  # the context is as good as before
    want, bound = ops_check.attention(q, k, v, [0, 300, 700], D ** -0.5)
    ops_check.within(out, want, bound)
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("H,D,T", [(64, 128, 1200), (40, 256, 900)])
def test_rows_computed_one_by_one_are_waited_for(xq, dtype, H, D, T):  # noqa: F811
    """A warp has up to 32 rows by itself, some 10^7 clocks, in each of many items: what
    the limit has beside the short time. No row may be lost."""
    assert xq.device_error() == 0
    q, k, v = inputs(T, H, 1, D, dtype, 42)
    v[0, 0, 9] = float("nan")
    s = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = xq.debug_stalled_prompt_attn(q, k, v, s, SHORT, False, out=torch.full_like(q, 7.0))
    assert xq.device_error() == 0
    want, bound = ops_check.attention(q, k, v, [0, T], D ** -0.5)
    assert bool(torch.isnan(out[..., 9]).all())
    want[..., 9] = math.nan
    ops_check.within(out, want, bound)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_long_search_is_waited_for(xq, dtype):  # noqa: F811
    """200000 sequences, most of them empty: looking for the first rows takes some 10^6 clocks."""
    assert xq.device_error() == 0
    n, lens = 200_000, [130, 1, 700]
    q, k, v = inputs(sum(lens), 2, 1, 64, dtype, 43)
    starts = torch.zeros(n + 1, dtype=torch.int32)
    at = 0
    for place, length in zip((7, 100_000, n - 1), lens):
        at += length
        starts[place + 1:] = at
    out = xq.debug_stalled_prompt_attn(q, k, v, starts.cuda(), SHORT, False)
    assert xq.device_error() == 0
    want, bound = ops_check.attention(q, k, v, [0, 130, 131, 831], 64 ** -0.5)
    ops_check.within(out, want, bound)
