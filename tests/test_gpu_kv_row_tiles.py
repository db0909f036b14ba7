"""Cache attention of 64 to 128 rows a KV head, which take one row tile with two buffers of scores, and its exactness."""
import pytest
import torch

import kv_oracle as ko
from test_gpu_kv_cache import attention_case, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


# At least 64 rows and 3 million rows x keys x KV heads; pages of one, two, four and eight 16-key groups; ragged ends.
@pytest.mark.parametrize("kind,dtype,heads,group,dim,page,n_q,prefix,lens", [
    ("q8", "bf16", 8, 4, 128, 64, 1, 3001, [1 + i % 9 for i in range(32)]),
    ("q8", "fp16", 8, 4, 128, 64, 1, 3001, [1 + i % 9 for i in range(32)]),
    ("q4", "fp16", 4, 5, 64, 16, 1, 8003, [i % 4 for i in range(20)]),
    ("q8", "fp16", 2, 11, 96, 32, 1, 23017, [5, 0, 40, 3, 2, 1]),
    ("q4", "bf16", 8, 9, 128, 128, 2, 5311, [9, 2, 1, 300]),
    ("q4", "fp16", 3, 100, 128, 32, 3, 3500, [4])])  # 300 rows: two chunks, the second with one row tile
def test_shared_prefix_on_one_row_tile(xq, kind, dtype, heads, group, dim, page, n_q, prefix, lens):  # noqa: F811
    attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, prefix=prefix, seed=prefix)


@pytest.mark.parametrize("kind,dtype,heads,group,dim,page,n_q,lens,window", [
    ("q8", "fp16", 4, 1, 128, 64, 65, [4500, 64, 0, 65], 0),
    ("q4", "bf16", 4, 1, 64, 16, 127, [2900, 2000, 126], 0),
    ("q8", "bf16", 4, 1, 96, 128, 65, [4500, 3064, 3066, 1], 3000)])
def test_own_pages_on_one_row_tile(xq, kind, dtype, heads, group, dim, page, n_q, lens, window):  # noqa: F811
    attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, window=window, seed=n_q)


@pytest.mark.parametrize("kind,heads,group,page,prefix,batch", [("q4", 2, 6, 32, 6001, 48), ("q8", 8, 4, 64, 4097, 64),
                                                                ("q8", 8, 4, 64, 20000, 4)])
def test_fp32_is_as_exact_as_fp32_arithmetic(xq, kind, heads, group, page, prefix, batch):  # noqa: F811
    """Root mean square error against 64 bits: at most twice that of the same operator in fp32 operations (both have fp32
    scores and sums; the kernels' operands have 22 bits of 24)."""
    dim, gen = 128, torch.Generator("cuda").manual_seed(prefix)
    pages = -(-prefix // page)
    cache = xq.KVCache({"q8": ko.Q8_0, "q4": ko.Q4_0}[kind], pages + batch, page, heads, dim)
    slots = torch.arange((pages + batch) * page, device="cuda")
    x = torch.randn(2, len(slots), heads, dim, device="cuda", generator=gen)
    cache.write(x[0], x[1], slots)
    q = torch.randn(batch, 1, heads * group, dim, device="cuda", generator=gen)
    table = torch.arange(pages, pages + batch, dtype=torch.int32, device="cuda").view(batch, 1)
    lens = torch.full((batch,), 5, dtype=torch.int32, device="cuda")
    out = cache.attn_shared(q, torch.arange(pages, dtype=torch.int32, device="cuda"), prefix, table, lens)
    k, v = cache.read(slots)
    error, plain, size = 0.0, 0.0, 0.0
    for b in range(batch):
        at = torch.cat((slots[:prefix], (pages + b) * page + torch.arange(5, device="cuda")))

        def attention(t):
            s = torch.einsum("hgd,lhd->hgl", q[b, 0].to(t).view(heads, group, dim), k[at].to(t)) * dim ** -0.5
            return torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), v[at].to(t)).reshape(-1, dim).double()
        want = attention(torch.float64)
        error += float(((out[b, 0].double() - want) ** 2).sum())
        plain += float(((attention(torch.float32) - want) ** 2).sum())
        size += float((want ** 2).sum())
    print((error / size) ** 0.5, (plain / size) ** 0.5)
    assert error <= 4 * plain, ((error / size) ** 0.5, (plain / size) ** 0.5)
