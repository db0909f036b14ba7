"""Adapters with infinities and NaN in x, A and B: what the definition gives, and no other row touched."""
import math

import pytest
import torch

from test_gpu_lora import adapters, some_ids, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
INF = math.inf


def agree(got, want):
    """Not finite in the same places: NaN, and infinities of the same sign."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    infinite = torch.isinf(want)
    assert torch.equal(torch.isinf(got), infinite) and torch.equal(got[infinite].sign(), want[infinite].sign().to(got.dtype))


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,rank,K,N", [(1, 8, 512, 64), (20, 16, 4096, 260), (90, 128, 512, 77), (700, 24, 96, 130), (2600, 64, 512, 264),
                                        (2500, 256, 96, 130)])
@pytest.mark.parametrize("where", ["x", "x mixed", "a", "b", "scale", "nan"])
def test_infinities(xq, dtype, M, rank, K, N, where):  # noqa: F811
    """x, A and B of small whole numbers, which one number of two holds exactly: the other is 0. Signs of A and B chosen so that
    infinities meet their like in some columns and their opposite in others."""
    g = torch.Generator("cuda").manual_seed(51)
    n = 3
    a, b, s = adapters(n, rank, K, N, dtype, 52)
    whole = lambda t: torch.randint(1, 8, t.shape, device="cuda", generator=g).to(t.dtype)  # noqa: E731
    a, b, s = whole(a), whole(b), whole(s)
    b[:, ::3] *= -1                     # columns that are infinite the other way
    b[:, 1::3, ::2] *= -1               # and such where infinities meet their opposite
    x, y = whole(torch.empty(M, K)).cuda(), torch.randn(M, N, device="cuda", generator=g)
    ids = some_ids(M, n, idle=False)
    ids[0] = 0
    clean = xq.Adapters([(a, b, s, 0)]).add([x], [y.clone()], ids)[0]
    hit = ids == 0
    if where.startswith("x"):
        x[0, 5] = INF
        if where == "x mixed":
            x[0, 6], x[0, K - 1] = 1.2345678, INF
        hit = torch.arange(M, device="cuda") == 0
    elif where == "a":
        a[0, 3, 7] = INF
    elif where == "b":
        b[0, N // 2, rank - 1] = INF
        b[0, 3, 0] = -INF
    elif where == "scale":
        s[0] = INF
    else:
        x[0, 0] = float("nan")
        a[0, 1, K - 1] = -INF
    got = xq.Adapters([(a, b, s, 0)]).add([x], [y.clone()], ids)[0]
    torch.cuda.synchronize()
    assert torch.equal(got[~hit], clean[~hit])
    rows = torch.nonzero(hit)[:, 0]
    t = (x[rows].double() @ a[0].double().T) * s[0].double()
    want = y[rows].double() + torch.stack([(t * b[0, c].double()).sum(-1) for c in range(N)], 1)
    agree(got[rows], want)
    finite = torch.isfinite(want)
    # sums of fp32 whose terms may be cut off: 2^-23 of the sum of magnitudes for each, K + rank + 8 of them
    size = (x[rows].double().abs() @ a[0].double().abs().T) * s[0].double() @ b[0].double().abs().T
    off = (got[rows].double() - want).abs() <= size * (K + rank + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -24
    assert bool(off[finite].all())
    assert xq.device_error() == 0
