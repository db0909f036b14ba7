"""Cache attention of 16-bit queries, held to what its arithmetic costs: which keys each row takes, key by key, and root mean
square errors of random data."""
import numpy as np
import pytest
import torch

import kv_check as kc
from test_gpu_kv_cache import rows, xq  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu

# (type, KV heads, query heads a KV head, dim, page, query tokens, own tokens of each sequence, window, prefix)
TILES = [
    ("q8", 8, 4, 128, 64, 1, [1 + i % 9 for i in range(32)], 0, 3001),     # 128 rows: one row tile
    ("q8", 2, 4, 128, 64, 1, [1 + i % 9 for i in range(128)], 0, 3001),    # 512 rows: two, twice
    ("q4", 2, 5, 64, 32, 1, [i % 4 for i in range(100)], 0, 3111),         # 500 rows
    ("q8", 1, 13, 96, 16, 3, [5, 0, 40, 3, 2, 1] * 3, 0, 6000),            # rows that end inside the prefix
    ("q4", 2, 3, 128, 128, 1, [7] * 64, 0, 8200),                          # 192 rows: one and a half
    ("q4", 3, 100, 128, 32, 3, [4], 0, 3500),                              # 300 rows of one sequence
    ("q8", 2, 4, 128, 64, 300, [1400, 299, 1, 0, 777], 0, 0),
    ("q4", 1, 7, 64, 16, 129, [2100, 129, 600], 0, 0),
    ("q8", 4, 1, 128, 64, 65, [4500, 64, 0, 65], 0, 0),
    ("q4", 2, 2, 96, 32, 400, [1003, 2050], 700, 0),
    ("q8", 4, 1, 96, 128, 65, [4500, 3064, 3066, 1], 3000, 0),
    ("q8", 2, 8, 64, 64, 2, [2 + i % 7 for i in range(64)], 0, 4111),
    ("q8", 1, 5, 96, 64, 1, [3] * 110, 0, 16100)]
SPLIT = [
    ("q8", 8, 4, 128, 16, 1, [1, 0, 15, 16, 17, 63, 64, 65, 130, 257], 0, 0),
    ("q4", 1, 16, 64, 16, 1, [1000, 33, 2], 0, 0),
    ("q8", 1, 6, 128, 32, 5, [5, 1, 205, 0, 41], 0, 0),
    ("q4", 2, 4, 256, 32, 3, [3, 700, 1], 0, 0),
    ("q8", 2, 4, 64, 16, 4, [3, 49, 200, 333], 50, 0),
    ("q8", 2, 4, 128, 32, 1, [1, 0, 17, 5], 0, 1000),
    ("q4", 1, 2, 96, 16, 9, [9, 20, 3, 0, 64], 0, 513)]
IDS = lambda c: "-".join(str(x if not isinstance(x, list) else len(x)) for x in c)  # noqa: E731


class Case:
    """A cache filled for a case's prefix and sequences (unwritten slots hold NaN scales), and its calls."""

    def __init__(self, xq, case, k, v, seed=0):  # noqa: F811
        kind, heads, _, dim, page, self.n_q, self.lens, self.window, self.prefix = case
        head, need = -(-self.prefix // page), [-(-n // page) for n in self.lens]
        pages = head + sum(need) + 1
        order = np.random.default_rng(seed).permutation(pages).astype(np.int32)
        table = np.full((len(need), max(need + [1]) + 1), -7, np.int32)
        at = head
        slots = [order[t // page] * page + t % page for t in range(self.prefix)]
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            slots += [table[b, t // page] * page + t % page for t in range(self.lens[b])]
            at += n
        self.xq, self.scale = xq, dim ** -0.5
        self.cache = xq.KVCache(kc.TYPES[kind], pages, page, heads, dim)
        self.cache.k.fill_(255)
        self.cache.v.fill_(255)
        slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        self.cache.write(k, v, slots)
        self.k, self.v = self.cache.read(slots)  # prefix, then each sequence's own
        self.pre, self.table = torch.from_numpy(order[:head]).cuda(), torch.from_numpy(table).cuda()

    def run(self, q, scale=None):
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan"))
        if self.prefix:
            self.cache.attn_shared(q, self.pre, self.prefix, self.table, lens, scale=scale, out=out)
        else:
            self.cache.attn(q, self.table, lens, scale=scale, window=self.window, out=out)
        assert self.xq.device_error() == 0
        return out

    def keys(self, b):
        """Indices into k and v of sequence b's keys, and which of them each query token sees."""
        first = self.prefix + sum(self.lens[:b])
        at = torch.cat((torch.arange(self.prefix), torch.arange(first, first + self.lens[b]))).cuda()
        return at, kc.seen(self.n_q, self.lens[b], self.window, self.prefix)

    def want(self, q, scale=None):
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for b in range(len(self.lens)):
            at, mask = self.keys(b)
            out[b] = kc.attention64(q[b], self.k[at], self.v[at], self.scale if scale is None else scale, mask)
        return out


def random_case(xq, case, dtype, seed=3):  # noqa: F811
    _, heads, group, dim, _, n_q, lens, _, prefix = case
    rng = np.random.default_rng(seed)
    total = prefix + sum(lens)
    k, v = (rows(rng, (total, heads, dim), "fp32").cuda() for _ in range(2))
    q = rows(rng, (len(lens), n_q, heads * group, dim), "fp32").to(kc.DTYPES[dtype]).cuda()
    return Case(xq, case, k, v), q


@gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", TILES + SPLIT, ids=IDS)
def test_root_mean_square_errors(xq, case, dtype):  # noqa: F811
    c, q = random_case(xq, case, dtype)
    want, out = c.want(q), c.run(q)
    assert kc.relative(out, want) <= kc.LIMIT[dtype], kc.relative(out, want)


@gpu
@pytest.mark.parametrize("case", TILES, ids=IDS)
def test_fp16_scores_keep_both_pieces_of_k(xq, case):  # noqa: F811
    """Queries four times larger: scores of some 10, where K as one fp16 number (2e-4) would cost 2e-3. With two pieces the
    scores are exact to fp32's rounding, and the limit stays that of ordinary scores."""
    c, q = random_case(xq, case, "fp16")
    q = q * 4
    want, out = c.want(q), c.run(q)
    assert kc.relative(out, want) <= kc.LIMIT["fp16"], kc.relative(out, want)


@gpu
@pytest.mark.parametrize("case", TILES, ids=IDS)
def test_fp16_outputs_keep_both_pieces_of_v(xq, case):  # noqa: F811
    """Queries of 0: all weights are one power of two, so the output's own rounding is all there is. V as one fp16 number would
    cost as much again, 1.4 times the error; half of that is allowed."""
    c, q = random_case(xq, case, "fp16")
    want, out = c.want(q * 0), c.run(q * 0)
    rounding = kc.relative(want.half(), want)
    assert kc.relative(out, want) <= 1.2 * rounding, (kc.relative(out, want), rounding)


# ------------------------------------------------------------ key by key

def marker_rounds(n, n_q, window, dim):
    """Sets of `dim` keys (fewer if there are not as many): the first and the last ones, every query token's own and the one
    after, the first that each row's window leaves and the one before, steps of 16 and 64, and some at random."""
    rng = np.random.default_rng(n)
    rounds = [np.arange(dim), n - 1 - np.arange(dim), 64 * np.arange(dim) - np.arange(dim) % 2, rng.integers(0, n, dim),
              16 * np.arange(dim) - np.arange(dim) % 2]
    rounds += [n - n_q + at + np.arange(dim) for at in range(0, n_q, dim)]
    if window:
        rounds += [n - n_q - window + at + np.arange(dim) for at in range(0, n_q + 1, dim)]
    return [np.unique(r[(r >= 0) & (r < n)]) for r in rounds]


def marked(total, heads, dim, marks, device="cuda"):
    """V rows that are 1 in element i of key marks[i] and 0 elsewhere."""
    v = torch.zeros(total, heads, dim, device=device)
    v[torch.as_tensor(marks, device=device), :, torch.arange(len(marks), device=device)] = 1
    return v


# An element is the marked key's value (as read back) over the number of keys, or exactly 0. Relative errors: the output's
# rounding (2^-11 or 2^-8); the weight as an fp16 number (2^-11); for bf16, V as one (2^-11); fp32 sums and quotients (2^-20).
KEY_LIMIT = {"fp16": 2 * 2.0 ** -11 + 2.0 ** -20, "bf16": 2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -20, "fp32": 2.0 ** -20}


def means(v, mask, heads, group):
    """float64 [n_q, heads * group, dim]: mean of the rows of v that each query token sees (0 if none)."""
    count = mask.sum(1).clamp(min=1).double()
    m = torch.einsum("il,lhd->ihd", mask.double(), v.double()) / count[:, None, None]
    return m.repeat_interleave(group, 1)


def off(got, want, dtype):
    return (got.double() - want).abs() > KEY_LIMIT[dtype] * want.abs()


@gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("case", TILES + SPLIT, ids=IDS)
def test_every_row_takes_its_keys_and_no_others(xq, case, dtype):  # noqa: F811
    """Queries of 0 give equal weights; V marks some keys, one an element."""
    _, heads, group, dim, _, n_q, lens, window, prefix = case
    total = prefix + sum(lens)
    longest = int(np.argmax(lens))
    k = torch.randn(total, heads, dim, device="cuda")
    q = torch.zeros(len(lens), n_q, heads * group, dim, dtype=kc.DTYPES[dtype], device="cuda")
    n = prefix + lens[longest]
    for marks in marker_rounds(n, n_q, window, dim):
        # keys of the longest sequence: the prefix's, and its own, which lie after those of the sequences before it
        at = np.where(marks < prefix, marks, marks + sum(lens[:longest]))
        c = Case(xq, case, k, marked(total, heads, dim, at))
        out = c.run(q)
        for b in range(len(lens)):
            keys, mask = c.keys(b)
            want = means(c.v[keys], mask, heads, group)
            assert not bool(off(out[b], want, dtype).any()), (b, marks[:4])


def test_the_key_by_key_limits_see_single_mistakes():
    """Mistakes planted in the definition: one key too many at the causal edge, all keys one too early, a 16-key step or a
    64-key tile left out."""
    n, n_q, window, dim = 3000, 70, 900, 64
    right = kc.seen(n_q, n, window, device="cpu")
    late = kc.seen(n_q, n + 1, window + 1, device="cpu")[:, :n]
    early = torch.cat((torch.zeros(n_q, 1, dtype=torch.bool), right[:, :-1]), 1)
    step, tile = right.clone(), right.clone()
    step[:, 2512:2528] = False
    tile[:, 2560:2624] = False
    rounds = [marked(n, 1, dim, m, "cpu") for m in marker_rounds(n, n_q, window, dim)]
    for dtype in KEY_LIMIT:
        want = [means(v, right, 1, 1) for v in rounds]
        for wrong in (late, early, tile):
            bad = torch.zeros(n_q, dtype=torch.bool)
            for v, w in zip(rounds, want):
                bad |= off(means(v, wrong, 1, 1), w, dtype).any(2).any(1)
            assert bad[(wrong != right).any(1)].all(), dtype
        assert any(bool(off(means(v, step, 1, 1), w, dtype).any()) for v, w in zip(rounds, want)), dtype


@gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [0.05, -0.05])
def test_row_tiles_with_bad_pages_and_odd_scales_within_rounding(xq, dtype, scale):  # noqa: F811
    """Pages without an id, V blocks from 1e-3 to 1e3 along the keys and 1e-2 to 1e2 along the elements, both signs of the
    scale. Errors by element group of 32, so that a block of small values answers for itself."""
    heads, group, dim, page, n, batch = 2, 8, 64, 16, 2000, 256
    rng = np.random.default_rng(12)
    cache = xq.KVCache(8, 126, page, heads, dim)
    k = rows(rng, (n, heads, dim), "fp32")
    v = rows(rng, (n, heads, dim), "fp32") * torch.logspace(-3, 3, n)[rng.permutation(n)][:, None, None] * torch.logspace(-2, 2, dim)
    slots = torch.arange(n, device="cuda")
    cache.write(k.cuda(), v.cuda(), slots)
    kf, vf = cache.read(slots)
    pre = torch.arange(125, dtype=torch.int32)
    keep = torch.ones(n, dtype=torch.bool)
    for p, bad in ((3, -1), (77, 126), (124, 1 << 30)):
        pre[p] = bad
        keep[p * page:(p + 1) * page] = False
    q = rows(rng, (batch, 1, heads * group, dim), "fp32").to(kc.DTYPES[dtype]).cuda()
    table, lens = torch.zeros(batch, 1, dtype=torch.int32, device="cuda"), torch.ones(batch, dtype=torch.int32, device="cuda")
    xq.device_error()
    out = cache.attn_shared(q, pre.cuda(), n, table, lens, scale=scale)
    assert xq.device_error() == (3 << 8) | 2
    kk, vv = torch.cat((kf[keep], kf[:1])), torch.cat((vf[keep], vf[:1]))
    want = torch.stack([kc.attention64(q[b], kk, vv, scale, torch.ones(1, len(kk), dtype=torch.bool, device="cuda")) for b in range(batch)])
    for d in range(0, dim, 32):
        a, w = out[..., d:d + 32], want[..., d:d + 32]
        past = w.abs() > 65504 * (1 + 2 ** -11) if dtype == "fp16" else torch.zeros_like(w, dtype=torch.bool)  # some large ones
        assert torch.isinf(a[past]).all() and int(past.sum()) < past.numel() // 100
        a, w = a[~past], w[~past]
        assert kc.relative(a, w) <= kc.LIMIT[dtype], (d, kc.relative(a, w))
