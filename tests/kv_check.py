"""What the cache attention's GPU tests share: a cache filled from given rows, the operator in 64 bits, relative errors."""
import torch

import kv_oracle as ko

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TYPES = {"q8": ko.Q8_0, "q4": ko.Q4_0}

# Root mean square error of an attention output over its root mean square. Rounding a number to 11 bits costs 2.1e-4 in that
# measure (a uniform error of half a step, 2^-11 of numbers from 1 to 2), to 8 bits 1.7e-3.
#   fp16: the output's rounding, and a softmax weight's as one fp16 number, which the sum of weights does not share: at most
#         2.9e-4 where one key takes all the weight. Together 3.6e-4; K, V and queries are exact. Limit 6e-4.
#   bf16: the output's rounding, weights and V as fp16 numbers, and K as fp16 numbers, which moves a score of size s by some
#         2e-4 s: for scores up to 5, 1e-3. Together 2.0e-3. Limit 4e-3.
#   fp32: two numbers of 22 bits in all for queries and weights, fp32 sums: as fp32 operations, 4e-7. Limit 2e-6.
LIMIT = {"fp32": 2e-6, "fp16": 6e-4, "bf16": 4e-3}

# (kernel, type, KV heads, query heads a KV head, query tokens, tokens): 64 and more 16-bit rows with 3 million rows x keys x
# heads take the tcgen05 tiles; what is smaller, and fp32, the split kernel, whose row forms these sizes select.
RUNS = [("tiles", "bf16", 2, 8, 128, 2000), ("tiles", "fp16", 2, 8, 128, 2000), ("tiles", "fp16", 8, 1, 96, 5000),
        ("split", "fp32", 2, 3, 20, 300), ("split", "fp16", 2, 3, 20, 300), ("split", "bf16", 2, 2, 2, 700),
        ("split", "fp32", 1, 1, 3, 5000)]


def filled(xq, kind, k, v, page, seed=0):
    """A cache that holds the rows k, v [n, heads, dim] (fp32, CUDA) in scattered pages, and the page table [1, pages]."""
    n, heads, dim = k.shape
    pages = -(-n // page)
    gen = torch.Generator().manual_seed(seed)
    table = torch.randperm(pages + 3, generator=gen)[:pages].to(torch.int32).cuda()
    cache = xq.KVCache(TYPES[kind], pages + 3, page, heads, dim)
    t = torch.arange(n, device="cuda")
    slots = table[t // page].long() * page + t % page
    cache.write(k, v, slots)
    return cache, table[None], slots


def seen(n_q, n, window=0, prefix=0, device="cuda"):
    """bool [n_q, prefix + n]: which keys each query token sees."""
    pos = torch.arange(prefix + n - n_q, prefix + n, device=device)[:, None]
    j = torch.arange(prefix + n, device=device)
    mask = j <= pos
    return mask & (j > pos - window) if window else mask


def attention64(q, k, v, scale, mask):
    """q [n_q, hq, dim] (any type), k and v [n, heads, dim], mask [n_q, n] -> float64 [n_q, hq, dim]; 0 for rows without a key.
    What is not finite in K or V counts as 0: callers look at rows that see none of it."""
    n_q, hq, dim = q.shape
    heads = k.shape[1]
    if k.shape[0] == 0:
        return torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    k, v = (torch.nan_to_num(x.double(), 0.0, 0.0, 0.0) for x in (k, v))
    z = torch.einsum("ihgd,lhd->hgil", q.double().view(n_q, heads, hq // heads, dim), k) * scale
    z = z.masked_fill(~mask, -float("inf"))
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -float("inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    return torch.einsum("hgil,lhd->ihgd", p, v).reshape(n_q, hq, dim)


def relative(got, want):
    """Root mean square error over the root mean square of `want`."""
    d = got.double() - want
    return float((d.square().sum() / want.square().sum()).sqrt())
