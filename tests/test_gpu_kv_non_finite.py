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
