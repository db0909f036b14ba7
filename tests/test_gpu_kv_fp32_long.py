"""fp32 cache attention over long runs of keys: the error does not grow with the length."""
import pytest
import torch

import kv_check as kc
from test_gpu_kv_cache import xq  # noqa: F401 (the fixture)
from test_gpu_kv_sharp import Case

pytestmark = pytest.mark.gpu


def attention32(q, k, v, scale, mask):
    """The operator in fp32 operations (products, exp, sums), as attention64 is in 64-bit ones."""
    n_q, hq, dim = q.shape
    heads = k.shape[1]
    z = torch.einsum("ihgd,lhd->hgil", q.view(n_q, heads, hq // heads, dim), k) * scale
    p = torch.softmax(z.masked_fill(~mask, -float("inf")), -1)
    return torch.einsum("hgil,lhd->ihgd", p, v).reshape(n_q, hq, dim)


# So many pairs of sequence and head that a CTA has thousands of keys of one: (type, KV heads, query heads a KV head, dim, page,
# query tokens, own tokens, window, prefix), factor of the queries.
@pytest.mark.parametrize("size", [0.1, 1.0, 3.0])
@pytest.mark.parametrize("case", [
    ("q8", 8, 4, 128, 64, 1, [5] * 64, 0, 32768), ("q4", 8, 4, 128, 64, 1, [5] * 40, 0, 17000),
    ("q8", 1, 5, 256, 32, 17, [17] * 30, 0, 17299), ("q4", 2, 3, 256, 64, 2, [9] * 64, 0, 9001),
    ("q8", 3, 1, 64, 64, 70, [70] * 12, 0, 20000), ("q8", 4, 4, 96, 16, 1, [7] * 50, 0, 12000),
    ("q8", 8, 4, 128, 64, 1, [20000, 17000] * 16, 0, 0)], ids=lambda c: "-".join(str(x if not isinstance(x, list) else x[0]) for x in c))
def test_as_exact_as_fp32_operations(xq, case, size):  # noqa: F811
    """Root mean square error against 64 bits: at most twice that of the same operator in fp32 operations."""
    _, heads, group, dim, _, n_q, lens, _, prefix = case
    gen = torch.Generator("cuda").manual_seed(prefix)
    total = prefix + sum(lens)
    k, v = (torch.randn(total, heads, dim, device="cuda", generator=gen) for _ in range(2))
    c = Case(xq, case, k, v)
    q = torch.randn(len(lens), n_q, heads * group, dim, device="cuda", generator=gen) * size
    out = c.run(q)
    error = plain = 0.0
    for b in range(0, len(lens), max(1, len(lens) // 4)):
        at, mask = c.keys(b)
        want = kc.attention64(q[b], c.k[at], c.v[at], c.scale, mask)
        error += float((out[b].double() - want).square().sum())
        plain += float((attention32(q[b], c.k[at], c.v[at], c.scale, mask).double() - want).square().sum())
    assert error <= 4 * plain, (error / plain) ** 0.5
