"""Keys whose stored blocks are not finite: only the rows that see them may notice."""
import numpy as np
import pytest
import torch

import kv_check as kc
from test_gpu_kv_cache import rows, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu
DIM, BLOCK = 64, 1  # the block of head 0 that is spoilt: elements 32 .. 63


def run(xq, kind, dtype, heads, group, n_q, n, what, value, at, window):  # noqa: F811
    """Attention over a cache in which one block of one key of head 0 is not finite: the output, the operator in 64 bits
    without that block, and which query tokens see the key."""
    rng = np.random.default_rng(n + at)
    k, v = (rows(rng, (n, heads, DIM), "fp32").cuda() for _ in range(2))
    (k if what == "k" else v)[at, 0, 32 * BLOCK + 7] = value
    cache, table, slots = kc.filled(xq, kind, k, v, 16)
    q = rows(rng, (1, n_q, heads * group, DIM), "fp32").to(kc.DTYPES[dtype]).cuda()
    out = cache.attn(q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), window=window)[0].float()
    mask = kc.seen(n_q, n, window)
    want = kc.attention64(q[0], *cache.read(slots), DIM ** -0.5, mask)
    assert xq.device_error() == 0
    return out, want, mask[:, at]


def places(n_q, n):
    """(key, window): the last token's key; one some way back; the same behind a short window that has passed it for the last
    rows; an early one that a long window (so that the tiles are taken) has passed for the second half of the rows; the first
    key that a window leaves to the first row."""
    return [(n - 1, 0), (n - n_q // 2 - 1, 0), (n - n_q // 2 - 1, max(1, n_q // 4)), (n // 8, n - n // 8 - n_q // 2),
            (n - n_q - n // 2 + 1, n // 2)]


def check_rows_beside_a_bad_key(xq, case, kind, what, value):  # noqa: F811
    _, dtype, heads, group, n_q, n = case
    for at, window in places(n_q, n):
        out, want, sees = run(xq, kind, dtype, heads, group, n_q, n, what, value, at, window)
        bad = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        bad[sees, :group] = True
        if what == "v":
            bad[..., :32 * BLOCK] = False
            bad[..., 32 * BLOCK + 32:] = False
        assert torch.equal(torch.isnan(out), bad), (at, window, int(torch.isnan(out).sum()), int(bad.sum()))
        good = ~bad
        assert kc.relative(out[good], want[good]) <= kc.LIMIT[dtype], (at, window, kc.relative(out[good], want[good]))


@pytest.mark.parametrize("case", kc.RUNS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("kind", ["q8", "q4"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_key_that_is_not_finite_is_for_the_rows_that_see_it(xq, case, kind, value):  # noqa: F811
    check_rows_beside_a_bad_key(xq, case, kind, "k", value)


@pytest.mark.parametrize("case", kc.RUNS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("kind", ["q8", "q4"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_value_that_is_not_finite_is_for_the_rows_that_see_it(xq, case, kind, value):  # noqa: F811
    check_rows_beside_a_bad_key(xq, case, kind, "v", value)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("prefix,batch,group", [(70, 3, 2), (3001, 24, 4)])  # (the second: bf16 on the tiles)
@pytest.mark.parametrize("what", ["k", "v"])
def test_behind_a_shared_prefix(xq, dtype, prefix, batch, group, what):  # noqa: F811
    """A bad block in one sequence's own tokens spoils that sequence alone; one in the prefix all of them."""
    heads, page, own = 8, 16, 5
    rng = np.random.default_rng(prefix)
    pages = -(-prefix // page)
    slots = torch.cat([torch.arange(prefix)] + [(pages + b) * page + torch.arange(own) for b in range(batch)]).cuda()
    q = rows(rng, (batch, 1, heads * group, DIM), "fp32").to(kc.DTYPES[dtype]).cuda()
    k, v = (rows(rng, (len(slots), heads, DIM), "fp32").cuda() for _ in range(2))
    for at, spoilt in ((prefix + own + 1, [1]), (prefix // 2, range(batch))):
        x = [k.clone(), v.clone()]
        x[what == "v"][at, 2, 32 * BLOCK] = float("inf")
        cache = xq.KVCache(8, pages + batch, page, heads, DIM)
        cache.write(*x, slots)
        out = cache.attn_shared(q, torch.arange(pages, dtype=torch.int32, device="cuda"), prefix,
                                torch.arange(pages, pages + batch, dtype=torch.int32, device="cuda")[:, None],
                                torch.full((batch,), own, dtype=torch.int32, device="cuda"))[:, 0].float()
        bad = torch.zeros_like(out, dtype=torch.bool)
        bad[list(spoilt), 2 * group:3 * group, slice(32 * BLOCK, 32 * BLOCK + 32) if what == "v" else slice(None)] = True
        assert torch.equal(torch.isnan(out), bad)
        kf, vf = cache.read(slots)
        for b in range(batch):
            j = torch.cat((torch.arange(prefix), prefix + own * b + torch.arange(own))).cuda()
            want = kc.attention64(q[b], kf[j], vf[j], DIM ** -0.5, kc.seen(1, own, prefix=prefix))[0]
            assert kc.relative(out[b][~bad[b]], want[~bad[b]]) <= kc.LIMIT[dtype]
        assert xq.device_error() == 0
