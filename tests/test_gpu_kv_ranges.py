"""Attention where the sizes of numbers are far apart or far from 1: the result depends on their ratios only."""
import numpy as np
import pytest
import torch

import kv_check as kc
from test_gpu_kv_cache import rows, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
DIM = 64
IDS = lambda c: "-".join(map(str, c))  # noqa: E731


def setup(case, seed=1):
    _, dtype, heads, group, n_q, n = case
    rng = np.random.default_rng(seed)
    k, v = (rows(rng, (n, heads, DIM), "fp32").cuda() for _ in range(2))
    q = rows(rng, (1, n_q, heads * group, DIM), "fp32").cuda()
    return k, v, q.to(kc.DTYPES[dtype]), torch.tensor([n], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("case", kc.RUNS, ids=IDS)
@pytest.mark.parametrize("kind", ["q8", "q4"])
def test_scales_far_below_the_largest(xq, kind, case):  # noqa: F811
    """One key in the middle has a K block 2^20 times the others' (in elements where every query is 0) and the last one V
    blocks 2^20 times the others': neither takes part in the earlier tokens' outputs, nor may it cost them bits."""
    _, dtype, heads, group, n_q, n = case
    k, v, q, lens = setup(case)
    q[..., 32:] = 0
    k, v, q = k / 32, v / 32, q * 32  # so that the large blocks' scales are fp16 numbers
    k[n // 2, :, 32:] *= 2.0 ** 20
    v[n - 1] *= 2.0 ** 20
    cache, table, slots = kc.filled(xq, kind, k, v, 32)
    out = cache.attn(q, table, lens)[0]
    want = kc.attention64(q[0], *cache.read(slots), DIM ** -0.5, kc.seen(n_q, n))
    assert kc.relative(out[:-1], want[:-1]) <= kc.LIMIT[dtype], kc.relative(out[:-1], want[:-1])
    assert xq.device_error() == 0


@pytest.mark.parametrize("case", kc.RUNS, ids=IDS)
@pytest.mark.parametrize("power", [-100, 90, 116, 120])
def test_queries_of_any_size(xq, case, power):  # noqa: F811
    """Queries times 2^x with a scale of 2^-x: the same scores."""
    _, dtype, heads, group, n_q, n = case
    k, v, q, lens = setup(case)
    if dtype == "fp16":
        power //= 12  # its range
    cache, table, slots = kc.filled(xq, "q8", k, v, 32)
    out = cache.attn(q * 2.0 ** power, table, lens, scale=DIM ** -0.5 * 2.0 ** -power)[0]
    want = kc.attention64(q[0], *cache.read(slots), DIM ** -0.5, kc.seen(n_q, n))
    assert kc.relative(out, want) <= kc.LIMIT[dtype], kc.relative(out, want)
    assert xq.device_error() == 0


@pytest.mark.parametrize("case", kc.RUNS, ids=IDS)
@pytest.mark.parametrize("power", [14, 18, 20, 21, 22, 23, 24, 26, 30])
def test_large_scores(xq, case, power):  # noqa: F811
    """Scores whose steps in fp32 are larger than a weight's range (16 at 2^27): the key with the largest one takes all the
    weight. V has scales above 1, which the split kernel's range follows too."""
    _, dtype, heads, group, n_q, n = case
    k, v, q, lens = setup(case)
    v = v * 256
    cache, table, slots = kc.filled(xq, "q8", k, v, 32)
    out = cache.attn(q, table, lens, scale=2.0 ** power)[0]
    kf, vf = cache.read(slots)
    want = kc.attention64(q[0], kf, vf, 2.0 ** power, kc.seen(n_q, n))
    # rows where the two largest scores are too close for the kernels' operands to tell apart are left out
    z = torch.einsum("ihgd,lhd->ihgl", q[0].double().view(n_q, heads, group, DIM), kf.double()).masked_fill(
        ~kc.seen(n_q, n)[:, None, None], -float("inf"))
    top = z.topk(2, -1).values
    clear = ((top[..., 0] - top[..., 1]) > 4e-3 * top[..., 0].abs()).reshape(n_q, heads * group)
    assert clear.any() and torch.isfinite(out).all()
    assert kc.relative(out[clear], want[clear]) <= kc.LIMIT[dtype], kc.relative(out[clear], want[clear])
    assert xq.device_error() == 0


@pytest.mark.parametrize("case", [c for c in kc.RUNS if c[1] != "fp16"], ids=IDS)
@pytest.mark.parametrize("size", [1e28, 1e30, 1e32])
def test_scores_far_below_zero(xq, case, size):  # noqa: F811
    """Every score is a large negative number: the key with the largest one still takes all the weight."""
    _, dtype, heads, group, n_q, n = case
    k, v, q, lens = setup(case)
    k = k.abs() + 0.1
    q = -(q.abs() + 0.1)
    cache, table, slots = kc.filled(xq, "q8", k, v, 32)
    out = cache.attn(q, table, lens, scale=size)[0]
    want = kc.attention64(q[0], *cache.read(slots), size, kc.seen(n_q, n))
    # rows where the two largest scores are too close for the kernels' operands to tell apart are left out
    kf = cache.read(slots)[0].double()
    z = torch.einsum("ihgd,lhd->ihgl", q[0].double().view(n_q, heads, group, DIM), kf).masked_fill(
        ~kc.seen(n_q, n)[:, None, None], -float("inf"))
    top = z.topk(2, -1).values
    clear = ((top[..., 0] - top[..., 1]) > 4e-3 * top[..., 0].abs()).reshape(n_q, heads * group)
    assert clear.any()
    assert kc.relative(out[clear], want[clear]) <= kc.LIMIT[dtype], kc.relative(out[clear], want[clear])
    assert xq.device_error() == 0


@pytest.mark.parametrize("case", [c for c in kc.RUNS if c[0] == "tiles"], ids=IDS)
def test_a_window_of_the_largest_size_is_no_window(xq, case):  # noqa: F811
    """Bit for bit: the same kernel has to be chosen."""
    k, v, q, lens = setup(case)
    cache, table, _ = kc.filled(xq, "q8", k, v, 32)
    out = cache.attn(q, table, lens)
    for window in (case[5], 2 ** 31 - 200, 2 ** 31 - 1):
        assert torch.equal(cache.attn(q, table, lens, window=window), out)
    assert xq.device_error() == 0
