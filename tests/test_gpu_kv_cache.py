"""The quantized KV cache on the GPU: stored bytes, read-back and attention against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import kv_oracle as ko

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TYPES = {"q8": ko.Q8_0, "q4": ko.Q4_0}


@pytest.fixture(scope="module")
def xq():
    from gguf_quant_integer_gb300 import build, xq as _xq
    build.build()
    _xq.lib()
    torch.cuda.synchronize()
    _xq.device_error()
    return _xq


def rows(rng, shape, dtype):
    """Random rows of dtype, as a CPU tensor."""
    x = rng.standard_normal(shape).astype(np.float32) * (1 + 6 * (rng.random(shape[-2:]) < 0.05)).astype(np.float32)
    return torch.from_numpy(x).to(DTYPES[dtype])


def make_cache(xq, kind, n_pages, page, heads, dim, fill=0xA5):
    c = xq.KVCache(TYPES[kind], n_pages, page, heads, dim)
    c.k.fill_(fill)
    c.v.fill_(fill)
    return c


# ------------------------------------------------------------- write, read

@pytest.mark.parametrize("kind", ["q8", "q4"])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("dim,heads,page,tokens,lead", [(128, 8, 64, 1, 0), (128, 2, 32, 77, 5), (64, 3, 16, 33, 0),
                                                        (96, 1, 128, 200, 3), (256, 2, 16, 19, 1)])
def test_write_stores_the_defined_bytes_and_read_returns_their_values(xq, kind, dtype, dim, heads, page, tokens, lead):
    rng = np.random.default_rng(dim + tokens)
    n_pages = -(-tokens // page) + 2
    cache = make_cache(xq, kind, n_pages, page, heads, dim)
    kp = ko.Pool(TYPES[kind], n_pages, page, heads, dim, 0xA5)
    vp = ko.Pool(TYPES[kind], n_pages, page, heads, dim, 0xA5)
    slots = rng.permutation(n_pages * page)[:tokens].astype(np.int64)
    # `lead` elements before K: rows that are not 16-byte aligned take the element-wise loads
    qkv = rows(rng, (tokens, 2 * heads, dim), dtype).reshape(tokens, -1)
    wide = torch.zeros((tokens, lead + 2 * heads * dim + lead), dtype=DTYPES[dtype])
    wide[:, lead:lead + 2 * heads * dim] = qkv
    wide = wide.cuda()
    k = wide[:, lead:lead + heads * dim].unflatten(1, (heads, dim))
    v = wide[:, lead + heads * dim:lead + 2 * heads * dim].unflatten(1, (heads, dim))
    drop = rng.random(tokens) < 0.2 if tokens > 1 else np.zeros(1, bool)
    given = np.where(drop, -1 - slots, slots)
    cache.write(k, v, torch.from_numpy(given).cuda())
    kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
    for t in np.nonzero(~drop)[0]:
        kp.put(int(slots[t]), kf[t])
        vp.put(int(slots[t]), vf[t])
    assert np.array_equal(cache.k.cpu().numpy(), kp.raw)  # and nothing else was written
    assert np.array_equal(cache.v.cpu().numpy(), vp.raw)
    for out in ("fp32", "fp16", "bf16"):
        gk, gv = cache.read(torch.from_numpy(given).cuda(), DTYPES[out])
        for got, pool in ((gk, kp), (gv, vp)):
            ref = pool.rows(np.where(drop, 0, slots))
            ref[drop] = 0
            # one rounding of the exact product: fp32 holds it, so the narrower types round the same number
            want = torch.from_numpy(ref.astype(np.float32)).to(DTYPES[out])
            assert torch.equal(got.cpu(), want)
    assert xq.device_error() == 0


@pytest.mark.parametrize("kind", ["q8", "q4"])
def test_write_edge_blocks(xq, kind):
    # zeros, ties, signs of the largest element, subnormal and huge scales, infinities and NaN
    top = 127.0 if kind == "q8" else 8.0
    x = np.zeros((12, 1, 64), np.float32)
    x[1, 0, :4] = [top, 0.5, -0.5, 1.5]              # d = 1 (or -1): exact halves
    x[2, 0, :4] = [-top, 2.5, -2.5, 3.4999]
    x[3, 0, 5], x[3, 0, 9] = 3.0, -3.0               # equal magnitudes: the first decides the sign
    x[4, 0, 9], x[4, 0, 5] = 3.0, -3.0
    x[5, 0, :32] = 1e-7 * np.arange(32)              # a subnormal scale
    x[6, 0, :32] = 1e-9                              # a scale that rounds to 0
    x[7, 0, :32] = np.linspace(-4e5, 4e5, 32)
    x[8, 0, 3] = np.inf                              # this block reads back as NaN, the next one does not
    x[9, 0, 40] = np.nan
    x[10, 0, :32] = np.linspace(-6e4, 6e4, 32)
    x[11] = np.random.default_rng(3).standard_normal((1, 64)) * 1e30
    cache = make_cache(xq, kind, 1, 16, 1, 64, 0)
    pool = ko.Pool(TYPES[kind], 1, 16, 1, 64)
    slots = torch.arange(12, device="cuda")
    t = torch.from_numpy(x).cuda()
    cache.write(t, t, slots)
    for s in range(12):
        pool.put(s, x[s])
    got, want = cache.k.cpu().numpy(), pool.raw
    nan = [1024 // (1 if kind == "q8" else 2) + 4 * 9 + 2 + i for i in (0, 1)]  # the NaN scale's bits are free
    keep = np.ones(got.size, bool)
    keep[nan] = False
    assert np.array_equal(got[keep], want[keep])
    k, _ = cache.read(slots)
    k = k.cpu().numpy()[:, 0]
    assert np.isnan(k[8, :32]).all() and np.array_equal(k[8, 32:], np.zeros(32))
    assert np.isnan(k[9, 32:]).all() and np.array_equal(k[9, :32], np.zeros(32))
    assert not np.isfinite(k[11]).any()
    assert np.isfinite(k[:8]).all()


def test_bad_slots_are_skipped_and_recorded(xq):
    cache = make_cache(xq, "q8", 2, 16, 1, 64, 7)
    before = cache.k.clone()
    x = torch.randn(2, 1, 64, device="cuda")
    cache.write(x, x, torch.tensor([32, -5], device="cuda"))
    assert xq.device_error() == (3 << 8) | 1
    assert torch.equal(cache.k, before)
    k, v = cache.read(torch.tensor([1 << 40, -1], device="cuda"))
    assert xq.device_error() == (3 << 8) | 1
    assert not k.any() and not v.any()
    assert xq.device_error() == 0


def test_pool_past_two_gigabytes(xq):
    # 64-bit offsets: the last page of a pool of 2.4 GB
    page, heads, dim = 64, 8, 128
    n_pages = 2_400_000_000 // (page * heads * dim * 34 // 32) + 1
    cache = xq.KVCache(ko.Q8_0, n_pages, page, heads, dim)
    rng = np.random.default_rng(8)
    x = rows(rng, (40, heads, dim), "fp32")
    slots = torch.arange((n_pages - 1) * page + 5, (n_pages - 1) * page + 45, device="cuda")
    cache.write(x.cuda(), x.cuda(), slots)
    k, v = cache.read(slots)
    codes, d = ko.quantize(x.numpy(), ko.Q8_0)
    want = ko.values(codes, d, ko.Q8_0).astype(np.float32)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want)
    q = rows(rng, (1, 1, 32, dim), "fp32")
    table = torch.full((1, 1), n_pages - 1, dtype=torch.int32, device="cuda")
    # keys 0..4 of the page are zeros as allocated
    out = cache.attn(q.cuda(), table, torch.tensor([45], dtype=torch.int32, device="cuda"))
    kk = np.concatenate((np.zeros((5, heads, dim)), want.astype(np.float64)))
    ref = ko.attention(q.numpy()[0], kk, kk, dim ** -0.5, [44])
    assert np.all(np.abs(out[0].cpu().numpy() - ref[0]) <= ko.tolerance(*ref, "fp32"))


# --------------------------------------------------------------- attention

def attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, window=0, prefix=0, seed=0, q_scale=1.0, poison=True):
    """A cache with one sequence per entry of lens (scattered pages), the call, and the oracle's answer."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    head = -(-prefix // page)
    n_pages = sum(need) + head + 1
    order = rng.permutation(n_pages)
    # bytes of unwritten slots: all ones make NaN scales, which must not be seen
    kp = ko.Pool(TYPES[kind], n_pages, page, heads, dim, 0xFF if poison else 0)
    vp = ko.Pool(TYPES[kind], n_pages, page, heads, dim, 0xFF if poison else 0)
    width = max(need + [1]) + 1
    table = np.full((len(lens), width), -7, np.int32)
    at = head
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    pre = order[:head].astype(np.int32)

    def slot(ids, t):
        return int(ids[t // page]) * page + t % page

    cache = xq.KVCache(TYPES[kind], n_pages, page, heads, dim, k=torch.from_numpy(kp.raw).cuda(), v=torch.from_numpy(vp.raw).cuda())
    slots = [slot(pre, t) for t in range(prefix)] + [slot(table[b], t) for b, n in enumerate(lens) for t in range(n)]
    k, v = rows(rng, (len(slots), heads, dim), "fp32"), rows(rng, (len(slots), heads, dim), "fp32")
    cache.write(k.cuda(), v.cuda(), torch.tensor(slots, dtype=torch.int64, device="cuda"))
    kp.raw, vp.raw = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    q = rows(rng, (len(lens), n_q, heads * group, dim), "fp32").mul(q_scale).to(DTYPES[dtype])
    args = (torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    if prefix:
        cache.attn_shared(q.cuda(), torch.from_numpy(pre).cuda(), prefix, *args, out=out)
    else:
        cache.attn(q.cuda(), *args, window=window, out=out)
    torch.cuda.synchronize()
    qf = q.float().numpy()
    pk, pv = kp.rows([slot(pre, t) for t in range(prefix)]), vp.rows([slot(pre, t) for t in range(prefix)])
    worst = 0.0
    for b, n in enumerate(lens):
        own = [slot(table[b], t) for t in range(n)]
        kk, vv = np.concatenate((pk, kp.rows(own))), np.concatenate((pv, vp.rows(own)))
        ref = ko.attention(qf[b], kk, vv, dim ** -0.5, [prefix + n - n_q + i for i in range(n_q)], window)
        got = out[b].float().cpu().numpy()
        assert np.isfinite(got).all(), b
        err, tol = np.abs(got - ref[0]), ko.tolerance(*ref, dtype)
        worst = max(worst, float((err / tol).max()))
        assert np.all(err <= tol), (b, n, float((err / tol).max()))
        assert not got[np.broadcast_to(ref[3] == 0, got.shape)].any()
    assert xq.device_error() == 0
    return worst


KINDS = [("q8", "fp32"), ("q8", "bf16"), ("q4", "fp16"), ("q4", "fp32")]


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("heads,group,dim", [(8, 4, 128), (2, 6, 128), (3, 1, 64), (1, 16, 64), (2, 5, 96), (1, 8, 256)])
def test_attention_of_single_tokens(xq, kind, dtype, heads, group, dim):
    # lengths around tiles and pages, none, one
    attention_case(xq, kind, dtype, heads, group, dim, 16, 1, [1, 0, 15, 16, 17, 63, 64, 65, 130, 257], seed=dim + heads)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("n_q,heads,group,dim", [(2, 2, 4, 128), (5, 1, 6, 128), (7, 2, 1, 64), (33, 1, 3, 96), (3, 1, 8, 256),
                                                 (150, 1, 2, 64), (40, 2, 4, 128)])
def test_attention_of_several_tokens_is_causal(xq, kind, dtype, n_q, heads, group, dim):
    # lens below n_q leave the first query tokens without a key
    attention_case(xq, kind, dtype, heads, group, dim, 32, n_q, [n_q, 1, n_q + 200, 0, 2 * n_q + 31], seed=n_q)


@pytest.mark.parametrize("kind,dtype", [("q8", "fp32"), ("q4", "bf16")])
@pytest.mark.parametrize("window", [1, 16, 50, 1000])
@pytest.mark.parametrize("n_q", [1, 4, 70])
def test_attention_window(xq, kind, dtype, window, n_q):
    attention_case(xq, kind, dtype, 2, 4, 64, 16, n_q, [3, 49, 200, 333], window=window, seed=window)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 7), (96, 1), (256, 2)])
@pytest.mark.parametrize("prefix,n_q,lens", [(100, 1, [1, 0, 17, 5]), (1, 2, [2, 3, 40]), (257, 1, list(range(1, 40))),
                                             (513, 9, [9, 20, 3, 0, 64])])
def test_shared_prefix(xq, kind, dtype, dim, group, prefix, n_q, lens):
    attention_case(xq, kind, dtype, 2, group, dim, 32, n_q, lens, prefix=prefix, seed=prefix + dim)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_large_scores_and_long_context(xq, dtype):
    # a few keys take all the weight; the running maximum moves along the sequence
    attention_case(xq, "q8", dtype, 1, 4, 128, 64, 1, [5000, 2777], seed=1, q_scale=20.0)
    attention_case(xq, "q8", dtype, 1, 4, 128, 64, 1, [20000], seed=2, q_scale=0.01)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shared", [False, True])
def test_values_of_very_different_sizes(xq, dtype, shared):
    # V blocks from 1e-4 to 1e4, the large ones late: the weights' working range has to follow
    heads, dim, page, n = 1, 64, 16, 300
    rng = np.random.default_rng(5)
    cache = xq.KVCache(ko.Q8_0, 32, page, heads, dim)
    k = rows(rng, (n, heads, dim), "fp32")
    v = rows(rng, (n, heads, dim), "fp32") * torch.logspace(-4, 4, n)[:, None, None]
    cache.write(k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
    q = rows(rng, (1, 1, 4, dim), "fp32").to(DTYPES[dtype])
    table = torch.arange(19, dtype=torch.int32, device="cuda")[None]
    if shared:
        out = cache.attn_shared(q.cuda(), table[0, :8].contiguous(), 128, table[:, 8:], torch.tensor([n - 128], dtype=torch.int32, device="cuda"))
    else:
        out = cache.attn(q.cuda(), table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    kf, vf = (t.cpu().numpy().astype(np.float64) for t in cache.read(torch.arange(n, device="cuda")))
    ref = ko.attention(q.float().numpy()[0], kf, vf, dim ** -0.5, [n - 1])
    assert np.all(np.abs(out[0].float().cpu().numpy() - ref[0]) <= ko.tolerance(*ref, dtype))


def test_bad_pages_and_lengths_are_masked_and_recorded(xq):
    heads, dim, page = 1, 64, 16
    rng = np.random.default_rng(6)
    cache = xq.KVCache(ko.Q8_0, 4, page, heads, dim)
    x = rows(rng, (64, heads, dim), "fp32")
    cache.write(x.cuda(), x.cuda(), torch.arange(64, device="cuda"))
    kf = cache.read(torch.arange(64, device="cuda"))[0].cpu().numpy().astype(np.float64)
    q = rows(rng, (1, 1, 4, dim), "fp32")

    def run(pages, n):
        return cache.attn(q.cuda(), torch.tensor([pages], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"))[0].cpu().numpy()

    def close(got, keys):
        ref = ko.attention(q.numpy()[0], keys, keys, dim ** -0.5, [len(keys) - 1])
        return np.all(np.abs(got - ref[0]) <= ko.tolerance(*ref, "fp32"))

    for bad in (4, -1, 2 ** 31 - 1):
        assert close(run([0, bad, 2], 40), np.concatenate((kf[:16], kf[32:40])))
        assert xq.device_error() == (3 << 8) | 2
    assert close(run([0, 1], 1000), kf[:32])
    assert xq.device_error() == (3 << 8) | 3
    assert not run([0, 1], -3).any()
    assert xq.device_error() == 0


def test_other_stream_and_own_workspace(xq):
    heads, dim, page, n = 2, 128, 32, 900
    rng = np.random.default_rng(7)
    cache = xq.KVCache(ko.Q4_0, 64, page, heads, dim)
    x = rows(rng, (n, heads, dim), "fp32").cuda()
    slots = torch.arange(n, device="cuda")
    q = rows(rng, (3, 1, 8, dim), "fp32").cuda()
    table = torch.arange(29, dtype=torch.int32, device="cuda").repeat(3, 1)
    lens = torch.tensor([900, 1, 512], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(q)
    cache.write(x, x, slots, stream=s)
    cache.attn(q, table, lens, out=out, stream=s)
    s.synchronize()
    again = cache.attn(q, table, lens)
    ws = torch.full((cache.attn_workspace_bytes(q.dtype, 3, 1, 8, 29),), 255, dtype=torch.uint8, device="cuda")
    third = cache.attn(q, table, lens, workspace=ws)
    # captured and replayed, on new queries
    g = torch.cuda.CUDAGraph()
    fixed = q.clone()
    with torch.cuda.graph(g):
        captured = cache.attn(fixed, table, lens, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(out, third) and torch.equal(out, captured)
    fixed.mul_(-1)
    g.replay()
    assert torch.equal(captured, cache.attn(-q, table, lens))


def test_repeated_calls_agree_bit_for_bit(xq):
    heads, dim, page = 2, 128, 16
    rng = np.random.default_rng(9)
    cache = xq.KVCache(ko.Q8_0, 300, page, heads, dim)
    x = rows(rng, (4800, heads, dim), "fp32").cuda()
    cache.write(x, x, torch.arange(4800, device="cuda"))
    table = torch.randperm(300, device="cuda").int().view(3, 100)
    lens = torch.tensor([1600, 77, 1003], dtype=torch.int32, device="cuda")
    pre = torch.arange(50, dtype=torch.int32, device="cuda")
    for dtype in DTYPES.values():
        q = torch.randn(3, 2, 12, dim, device="cuda").to(dtype)
        a, s = cache.attn(q, table, lens), cache.attn_shared(q, pre, 789, table, lens)
        for _ in range(5):
            assert torch.equal(cache.attn(q, table, lens), a)
            assert torch.equal(cache.attn_shared(q, pre, 789, table, lens), s)


# Enough rows x keys x KV heads for the tcgen05 tiles: 3 million a call for 16-bit queries, 8 million for fp32 ones (64 rows or more).

@pytest.mark.parametrize("kind,dtype,heads,group,dim,page,n_q,prefix,lens", [
    ("q8", "bf16", 2, 4, 128, 64, 1, 3001, [1 + i % 9 for i in range(128)]),
    ("q4", "fp16", 2, 5, 64, 32, 1, 3111, [i % 4 for i in range(100)]),           # 500 rows: a half-empty second tile
    ("q8", "fp16", 1, 13, 96, 16, 3, 6000, [5, 0, 40, 3, 2, 1] * 3),              # 702 rows; rows that end inside the prefix
    ("q4", "bf16", 2, 3, 128, 128, 1, 8200, [7] * 64),                            # 192 rows: one and a half row tiles
    ("q8", "fp32", 2, 8, 128, 64, 2, 4111, [2 + i % 7 for i in range(64)]),
    ("q4", "fp32", 2, 8, 64, 32, 1, 4000, [i % 3 for i in range(130)]),
    ("q8", "fp32", 1, 5, 96, 64, 1, 16100, [3] * 110)])
def test_shared_prefix_on_row_tiles(xq, kind, dtype, heads, group, dim, page, n_q, prefix, lens):
    attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, prefix=prefix, seed=prefix)


@pytest.mark.parametrize("kind,dtype,heads,group,dim,page,n_q,lens,window", [
    ("q8", "bf16", 2, 4, 128, 64, 300, [1400, 299, 1, 0, 777], 0),
    ("q4", "fp16", 1, 7, 64, 16, 129, [2100, 129, 600], 0),
    ("q4", "bf16", 2, 2, 96, 32, 400, [1003, 2050], 700),
    ("q8", "fp32", 2, 4, 128, 64, 333, [1800, 332, 40, 1111], 0),
    ("q4", "fp32", 1, 6, 64, 32, 257, [2600, 300, 2599], 1500)])
def test_long_query_runs_on_row_tiles(xq, kind, dtype, heads, group, dim, page, n_q, lens, window):
    attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, window=window, seed=n_q)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_row_tiles_with_bad_pages_and_odd_scales(xq, dtype):
    """Masked groups of a page without an id, V blocks from 1e-3 to 1e3, a negative scale of the scores."""
    heads, group, dim, page, n, rows_n = 2, 8, 64, 16, 2000, 128
    rng = np.random.default_rng(12)
    cache = xq.KVCache(ko.Q8_0, 126, page, heads, dim)
    k = rows(rng, (n, heads, dim), "fp32")
    v = rows(rng, (n, heads, dim), "fp32") * torch.logspace(-3, 3, n)[:, None, None] * torch.logspace(-2, 2, dim)
    cache.write(k.cuda(), v.cuda(), torch.arange(n, device="cuda"))
    kf, vf = (t.cpu().numpy().astype(np.float64) for t in cache.read(torch.arange(n, device="cuda")))
    pre = torch.arange(125, dtype=torch.int32)
    pre[3], pre[77], pre[124] = -1, 126, 1 << 30
    keep = np.ones(n, bool)
    for p in (3, 77, 124):
        keep[p * page:(p + 1) * page] = False
    n_q = 2 if dtype == "fp32" else 1
    q = rows(rng, (rows_n * 2, n_q, heads * group, dim), "fp32").to(DTYPES[dtype])
    table, lens = torch.zeros(rows_n * 2, 1, dtype=torch.int32, device="cuda"), torch.full((rows_n * 2,), n_q, dtype=torch.int32, device="cuda")
    xq.device_error()
    out = cache.attn_shared(q.cuda(), pre.cuda(), n, table, lens, scale=-0.05).float().cpu().numpy()
    assert xq.device_error() == (3 << 8) | 2
    for b in (0, 1, 100, 255):
        kk, vv = np.concatenate((kf[keep], kf[:n_q])), np.concatenate((vf[keep], vf[:n_q]))
        ref = ko.attention(q[b].float().numpy(), kk, vv, -0.05, [len(kk) - n_q + i for i in range(n_q)])
        err, tol = np.abs(out[b] - ref[0]), ko.tolerance(*ref, dtype)
        assert np.all(err <= tol), (b, float((err / tol).max()))
