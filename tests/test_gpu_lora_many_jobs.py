"""Adapters with more jobs than a launch has clusters (512): a cluster takes one after the other."""
import pytest
import torch

import ops_check
from test_gpu_lora import adapters, run, some_ids, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

# rows, adapters, rank, K, N: every row its own adapter; ranks whose sums are added up by each CTA, by shares of them, and both in
# turn (uneven numbers of rows); jobs of 16, 32 and 64 rows
SIZES = [(1000, 1000, 8, 64, 40), (1100, 1100, 128, 64, 33), (1000, 1000, 256, 32, 40), (2431, 2000, 8, 96, 36), (2431, 600, 256, 64, 30),
         (40000, 100, 16, 64, 40), (40000, 300, 8, 32, 17), (30000, 60, 256, 32, 40), (3000, 3000, 24, 64, 40)]


def uneven(M, n, seed=5):
    """Rows spread so that some adapters have many and most one or none."""
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(M, generator=g) ** 3 * n).to(torch.int32)
    ids[: M // 8] = torch.arange(M // 8, dtype=torch.int32) % n
    ids[::97] = -1
    return ids.cuda()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,n,rank,K,N", SIZES)
@pytest.mark.parametrize("spread", ["own", "uneven"])
def test_more_jobs_than_clusters(xq, dtype, M, n, rank, K, N, spread):  # noqa: F811
    ids = (torch.arange(M, dtype=torch.int32) % n)[torch.randperm(M, generator=torch.Generator().manual_seed(6))].cuda() if spread == "own" else uneven(M, n)
    p = adapters(n, rank, K, N, dtype, 61)
    g = torch.Generator("cuda").manual_seed(62)
    x, y = torch.randn(M, K, device="cuda", generator=g), torch.randn(M, N, device="cuda", generator=g)
    ad = xq.Adapters([(*p, 0)])
    got = ad.add([x], [y.clone()], ids)[0]
    # all rows at once: each row with its adapter
    a, b, s = (t.double() for t in p)
    want, bound = y.double(), torch.zeros_like(y, dtype=torch.float64)
    for first in range(0, M, 1000):
        rows = torch.arange(first, min(M, first + 1000), device="cuda")
        rows = rows[ids[rows] >= 0]
        i = ids[rows].long()
        t = torch.einsum("mk,mrk->mr", x[rows].double(), a[i])
        want[rows] += s[i, None] * torch.einsum("mr,mnr->mn", t, b[i])
        dt = torch.einsum("mk,mrk->mr", x[rows].double().abs(), a[i].abs()) * (2.0 ** -20 + (K + 8) * 2.0 ** -23)
        dt += t.abs() * (2.0 ** -20 + (rank + 8) * 2.0 ** -23)
        bound[rows] = s[i, None].abs() * torch.einsum("mr,mnr->mn", dt, b[i].abs()) + want[rows].abs() * 2.0 ** -24
    ops_check.within(got, want, bound)
    assert torch.equal(got[ids < 0], y[ids < 0])
    for _ in range(3):  # bit for bit the same
        assert torch.equal(ad.add([x], [y.clone()], ids)[0], got)
    assert xq.device_error() == 0


def test_many_jobs_of_projections_together(xq):  # noqa: F811
    """Two projections, one of fewer adapters than the ids name (recorded, the rest as ever)."""
    M = 1500
    ids = torch.arange(M, dtype=torch.int32, device="cuda")
    run(xq, M, [adapters(M, 16, 64, 40, "bf16", 1), adapters(700, 64, 96, 33, "bf16", 2)], ids)
    assert xq.device_error() == 5 << 8 | 1
