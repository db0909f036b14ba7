"""Prompt attention of fp32 rows whose sizes differ widely within 128 keys: as exact as ever, whatever a row's weights pick out."""
import pytest
import torch

import ops_check
from test_gpu_prompt_attn import inputs, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def check(xq, q, k, v, starts, scale=None, window=0):  # noqa: F811
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out = xq.prompt_attn(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale=scale, window=window)
    want, bound = ops_check.attention(q, k, v, starts, scale, window)
    ops_check.within(out, want, bound)
    assert xq.device_error() == 0
    return out, want


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -14, 2.0 ** 14, 2.0 ** 30])
@pytest.mark.parametrize("every", [1, 37, 400])
def test_single_rows_of_another_size(xq, D, size, every):  # noqa: F811
    """Ordinary rows, and single ones (keys, values, both) far smaller or larger."""
    T = 700
    q, k, v = inputs(T, 4, 2, D, "fp32", 71)
    for which in ("k", "v", "kv"):
        k2, v2 = k.clone(), v.clone()
        if "k" in which:
            k2[5::every if every > 1 else T] *= min(size, 2.0 ** 14)  # scores of 10^5 are as far as 64 bits are compared with 32
        if "v" in which:
            v2[5::every if every > 1 else T] *= size
        check(xq, q, k2, v2, [0, 300, T])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_values_that_have_no_weight(xq, D):  # noqa: F811
    """Values 2^24 and 2^40 times as large under keys whose weights are below 2^-60 of the others': the results are of the small ones,
    whose roundings (2^-24 of each, and 2^-39 of a value 2^40 as large would be 2) count. As exact as ordinary rows: the sums' errors at random, below
    1e-6 in the mean."""
    T = 600
    for size in (2.0 ** 13, 2.0 ** 24, 2.0 ** 40):
        q, k, v = inputs(T, 2, 1, D, "fp32", 72)
        q[..., 0] = 1.0
        k[..., 0] = 0.0
        far = torch.arange(T, device="cuda") % 5 == 3
        k[far, :, 0] = -100.0  # times the scale of 1: e^-100
        v[far] *= size
        out, want = check(xq, q * 0.1 + 0.9 * torch.nn.functional.one_hot(torch.zeros(1, dtype=torch.long, device="cuda"), D), k, v, [0, T], scale=1.0)
        rows = torch.arange(4, T, device="cuda")
        assert ops_check.rms(out[rows], want[rows]) <= 1e-6


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_keys_that_meet_small_queries(xq, D):  # noqa: F811
    """Keys far apart, and scores that are ordinary for the large ones, or for the small ones."""
    T = 500
    q, k, v = inputs(T, 2, 1, D, "fp32", 73)
    far = torch.arange(T, device="cuda") % 7 == 2
    k[far] *= 2.0 ** 20
    for power in (-20, -10, 0):
        out, want = check(xq, q * 2.0 ** power, k, v, [0, T])
        if power == -20:  # scores of a few at most
            assert ops_check.rms(out, want) <= 1.5e-6
