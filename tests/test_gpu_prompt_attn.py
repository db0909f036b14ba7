"""Causal attention over packed prompts, against 64 bits."""
import math

import pytest
import torch

import ops_check
from gguf_quant_integer_gb300 import build as xqbuild
from ops_check import DTYPES

pytestmark = pytest.mark.gpu

KINDS = ["fp32", "fp16", "bf16"]


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    return _xq


def inputs(T, H, Hk, D, dtype, seed=0, fused=False, spread=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(T, (H + 2 * Hk) * D, device="cuda", generator=g)
    x[:, :H * D] *= spread
    parts = x.to(DTYPES[dtype]).split([H * D, Hk * D, Hk * D], 1)
    q, k, v = parts if fused else [p.contiguous() for p in parts]
    return q.unflatten(1, (H, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))


def starts_of(lens, first=0):
    s = [first]
    for n in lens:
        s.append(s[-1] + n)
    return s


def case(xq, lens, H=4, Hk=2, D=128, dtype="bf16", window=0, scale=None, fused=False, first=0, behind=0, seed=0, spread=1.0):
    starts = starts_of(lens, first)
    T = starts[-1] + behind
    q, k, v = inputs(T, H, Hk, D, dtype, seed, fused, spread)
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, H, D), 7.0, dtype=q.dtype, device="cuda")
    xq.prompt_attn(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale=scale, window=window, out=out)
    torch.cuda.synchronize()
    assert xq.device_error() == 0
    want, bound = ops_check.attention(q, k, v, starts, scale, window)
    ops_check.within(out, want, bound, f"{lens} {H}/{Hk} {D} {dtype}")
    free = torch.isnan(want)
    assert bool((out[free] == 7.0).all())  # rows of no sequence are left as they were
    return q, k, v, starts, out, want


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("H,Hk,D", [(4, 1, 128), (7, 1, 64), (2, 2, 96), (6, 3, 256), (5, 1, 128), (16, 2, 64), (40, 1, 128), (3, 3, 256),
                                    (33, 1, 96)])
def test_lengths(xq, dtype, H, Hk, D):
    """Tiles of 128 rows and keys begin, end and are whole anywhere; sequences of none and one token."""
    case(xq, [1, 0, 2, 31, 33, 0, 64, 1, 127, 128, 129, 255, 257, 300], H, Hk, D, dtype, first=3, behind=5)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_longer_sequences(xq, dtype, D):
    case(xq, [1025, 700], 4, 2, D, dtype, fused=True)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 500, 2000, 1 << 31])
def test_windows(xq, dtype, window):
    case(xq, [777, 5, 300], 4, 2, 128, dtype, window=window)
    case(xq, [300, 129], 3, 1, 256, dtype, window=window)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("n", [1, 2, 16, 17])
def test_one_short_sequence(xq, dtype, n):
    case(xq, [n], 32, 8, 128, dtype)
    case(xq, [n], 1, 1, 64, dtype)


@pytest.mark.parametrize("dtype", KINDS)
def test_many_sequences(xq, dtype):
    case(xq, [(37 * i) % 23 for i in range(700)], 4, 2, 64, dtype)
    case(xq, [0] * 50 + [200] + [0] * 50 + [3], 2, 1, 128, dtype)


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.3, 1.0), (0.3, 8.0), (1.0, 30.0)])
def test_scales_and_sharp_scores(xq, dtype, scale, spread):
    """Scores from equal to hundreds apart: one key takes all. (Maxima that rise late move the softmax reference.)"""
    case(xq, [400, 130], 4, 2, 128, dtype, scale=scale, spread=spread)


@pytest.mark.parametrize("dtype", KINDS)
def test_rising_scores(xq, dtype):
    """Each later key scores higher than all before it, so every tile moves the reference."""
    T, D = 900, 128
    q, k, v = inputs(T, 2, 1, D, dtype, 5)
    q[:] = 1.0
    k[:, :, :] = (torch.arange(T, device="cuda").float() / T * 6)[:, None, None].to(k.dtype)
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    want, bound = ops_check.attention(q, k, v, [0, T], 1.0)
    ops_check.within(xq.prompt_attn(q, k, v, starts, scale=1.0), want, bound)


@pytest.mark.parametrize("dtype,limit", [("fp32", 1e-6), ("fp16", 4e-4), ("bf16", 3e-3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_root_mean_square(xq, dtype, limit, D):
    """Roundings at random: of 16-bit weights and of the result, each 0.41 of a half step (2^-11, 2^-8) in the mean; of fp32's
    sums some 4 of 2^-24."""
    *_, out, want = case(xq, [2048], 4, 2, D, dtype)
    assert ops_check.rms(out, want) <= limit


@pytest.mark.parametrize("dtype", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(xq, dtype, D, value):
    """Bad keys and values: behind the last sequence, in a later sequence and later in the same one."""
    q, k, v, starts, out, _ = case(xq, [200, 140, 61], 4, 2, D, dtype, behind=20, seed=3)
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for which in ("k", "v", "kv"):
        k2, v2 = k.clone(), v.clone()
        for x, name in ((k2, "k"), (v2, "v")):
            if name in which:
                x[starts[-1]:] = value       # no sequence's
                x[starts[1] + 100, 1, 5] = value  # row 100 of the second sequence, KV head 1
        got = xq.prompt_attn(q, k2, v2, s)
        same = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
        same[starts[1] + 100:starts[2], 2:] = False  # the rows that see it
        same[starts[-1]:] = False
        assert torch.equal(got[same], out[same])
        hit = got[starts[1] + 100:starts[2], 2:]
        if "v" in which:
            assert not bool(torch.isfinite(hit[..., 5]).any())
        elif math.isnan(value):
            assert bool(torch.isnan(hit).all())
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", KINDS)
def test_infinite_scores(xq, dtype):
    """A key that scores minus infinity has no weight (its other elements are 0, so that no product is NaN)."""
    T, D = 300, 64
    q, k, v = inputs(T, 2, 1, D, dtype, 9)
    q = q.abs() + 0.1
    k[7], k[150] = 0, 0
    k[7, 0, 3] = k[150, 0, 60] = -float("inf")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    got = xq.prompt_attn(q, k, v, starts)
    # 0 * q of the other elements is 0: the scores are minus infinity, not NaN
    k2, keep = k.clone(), torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[150] = False
    z = torch.einsum("ihd,jd->hij", q.double(), k2[:, 0].double()) * D ** -0.5
    z = z.masked_fill(~keep | (torch.arange(T, device="cuda")[:, None] < torch.arange(T, device="cuda")), -math.inf)
    want = torch.einsum("hij,jd->ihd", torch.softmax(z, -1), v[:, 0].double())
    assert bool(torch.isfinite(got).all())
    assert ops_check.rms(got, want) <= {"fp32": 2e-6, "fp16": 5e-4, "bf16": 4e-3}[dtype]


@pytest.mark.parametrize("dtype", KINDS)
def test_large_and_small_values(xq, dtype):
    """V near the type's end, scores past 2^20, rows of zeros."""
    T = 260
    q, k, v = inputs(T, 2, 1, 128, dtype, 11)
    v = v * (8000.0 if dtype == "fp16" else 2.0 ** 100)
    q[5] = 0
    q[77] *= 1000
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for scale in (0.1, 100000.0):
        got = xq.prompt_attn(q, k, v, starts, scale=scale)
        want, bound = ops_check.attention(q, k, v, [0, T], scale)
        # scores of 10^6 and more: fp32 scores may swap keys that lie nearer than their roundings; such rows are not looked at
        sharp = torch.isfinite(bound) & (bound < 0.5 * want.abs().amax(-1, keepdim=True)) if scale > 1 else torch.ones_like(bound, dtype=torch.bool)
        assert bool(torch.isfinite(got).all())
        ops_check.within(torch.where(sharp, got.double(), want), want, bound)


def test_bad_bounds_are_left_out_and_recorded(xq):
    q, k, v = inputs(300, 4, 2, 128, "bf16")
    good = torch.tensor([0, 100, 180, 300], dtype=torch.int32, device="cuda")
    want = xq.prompt_attn(q, k, v, good)
    assert xq.device_error() == 0
    for bad, live in (([0, 100, 90, 300], [(0, 90)]), ([-5, 100, 180, 300], [(100, 180), (180, 300)]), ([0, 100, 180, 301], [(0, 100), (100, 180)]),
                      ([0, 100, 2147483647, 300], [(0, 100)])):
        out = torch.full_like(want, 7.0)
        xq.prompt_attn(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out)
        assert xq.device_error() == 5 << 8 | 2
        for s, e in live:
            assert torch.equal(out[s:e], want[s:e])


@pytest.mark.parametrize("dtype", KINDS)
def test_rows_do_not_depend_on_the_batch(xq, dtype):
    """Alone, packed with others and packed again: bit for bit the same, as often as it is run."""
    q, k, v, starts, out, _ = case(xq, [130, 300, 17, 260], 8, 2, 128, dtype)
    for b in range(4):
        s = slice(starts[b], starts[b + 1])
        n = starts[b + 1] - starts[b]
        alone = xq.prompt_attn(q[s], k[s], v[s], torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        assert torch.equal(alone, out[s])
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    for _ in range(5):
        assert torch.equal(xq.prompt_attn(q, k, v, s), out)


@pytest.mark.parametrize("dtype", KINDS)
def test_streams_and_graphs(xq, dtype):
    q, k, v, starts, out, _ = case(xq, [400, 129], 4, 2, 128, dtype)
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = xq.prompt_attn(q, k, v, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, out)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(xq.prompt_attn(q, k, v, s, window=0 if i == 0 else 100))
        graphs.append(g)
    others = [torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda") for _ in range(100)]
    want = xq.prompt_attn(q, k, v, s, window=100)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], want) and all(bool((x == 7).all()) for x in others)
    s[1] = 300  # a replay goes by what starts holds then
    graphs[0].replay()
    assert torch.equal(outs[0], xq.prompt_attn(q, k, v, s))


def test_refusals_and_empty_calls(xq):
    q, k, v = inputs(10, 4, 2, 128, "bf16")
    s = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    ok = dict(q=q, k=k, v=v, starts=s)
    for kw in (dict(k=k[:9]), dict(v=v[:, :1]), dict(k=k.half()), dict(k=k.cpu()), dict(starts=s.long()), dict(starts=s[:0]), dict(starts=s.cpu()),
               dict(out=q[:9]), dict(out=q.float()), dict(q=q.double(), k=k.double(), v=v.double()),
               dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            xq.prompt_attn(**{**ok, **kw})
    for kw in (dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=q[:, :3].contiguous()),
               dict(q=q[..., :32].contiguous(), k=k[..., :32].contiguous(), v=v[..., :32].contiguous())):
        with pytest.raises(xq.XQError):
            xq.prompt_attn(**{**ok, **kw})
    with pytest.raises(xq.XQError):  # rows that are not 16 bytes' multiples apart
        x = torch.zeros(10, 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")
        xq.prompt_attn(x[:, :512].unflatten(1, (4, 128)), k, v, s)
    out = torch.full_like(q, 7.0)
    xq.prompt_attn(q, k, v, s[:1], out=out)
    assert bool((out == 7.0).all())
    assert xq.prompt_attn(q[:0], k[:0], v[:0], s).shape == (0, 4, 128)
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", KINDS)
def test_rows_computed_one_by_one(xq, dtype):
    """One bad element that all rows see: every row is computed by itself, its other elements as exactly as ever (fp32's sums; the
    weights are not rounded), over more keys than a step has and with a window."""
    T, D = 3000, 128
    q, k, v = inputs(T, 2, 1, D, dtype, 21)
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for window in (0, 77):
        v2 = v.clone()
        v2[::60, 0, 9] = float("nan")  # a window of 77 has at least one
        got = xq.prompt_attn(q, k, v2, starts, window=window)
        want, bound = ops_check.attention(q, k, v, [0, T], D ** -0.5, window)
        assert bool(torch.isnan(got[60:, :, 9]).all())
        want[:, :, 9] = math.nan
        ops_check.within(got, want, bound)
    assert xq.device_error() == 0


def test_rows_of_very_different_size(xq):
    """fp32 keys and values from 2^-40 to 2^60 beside each other, in the same 128 keys: each row as exact as its own sums allow."""
    T, D = 400, 128
    q, k, v = inputs(T, 2, 1, D, "fp32", 22)
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    size = 2.0 ** torch.linspace(-40, 60, T, device="cuda")[torch.randperm(T, device="cuda", generator=torch.Generator("cuda").manual_seed(1))]
    for kk, vv in ((k, v * size[:, None, None]), (k * (size[:, None, None] ** 0.05), v), (k * 1e-20, v * 1e-30), (k * 2.0 ** 100, v * 2.0 ** 100)):
        scale = D ** -0.5 / float(kk.abs().amax()) * 4
        got = xq.prompt_attn(q, kk.contiguous(), vv.contiguous(), starts, scale=scale)
        want, bound = ops_check.attention(q, kk, vv, [0, T], scale)
        ops_check.within(got, want, bound)
    # a channel far larger than the others
    v2 = v.clone()
    v2[:, :, 17] *= 1e9
    got = xq.prompt_attn(q, k, v2, starts)
    want, bound = ops_check.attention(q, k, v2, [0, T], D ** -0.5)
    assert ops_check.rms(got[..., :17], want[..., :17]) <= 1e-6 and ops_check.rms(got[..., 17], want[..., 17]) <= 1e-6
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_offsets_past_32_bits(xq, dtype):
    """More than 2^31 elements of q and of the result: the last sequence's rows, under a window."""
    H, D, lens = 32, 128, [524288 + 11, 700]
    T = sum(lens)
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.empty(T, H, D, dtype=DTYPES[dtype], device="cuda").normal_(generator=g)
    k, v = (torch.empty(T, 1, D, dtype=DTYPES[dtype], device="cuda").normal_(generator=g) for _ in range(2))
    s = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
    got = xq.prompt_attn(q, k, v, s, window=300)
    for a, e in ((lens[0] - 600, lens[0]), (lens[0], T)):
        want, bound = ops_check.attention(q[a:e], k[a:e], v[a:e], [0, e - a], D ** -0.5, 300)
        skip = 300 if a < lens[0] else 0  # rows whose window begins before the part that is compared
        ops_check.within(got[a + skip:e], want[skip:], bound[skip:])
    assert xq.device_error() == 0


def test_a_long_sequence(xq):
    """131071 keys: the last rows' sums over all of them."""
    T, D = 131071, 128
    for dtype, limit in (("bf16", 3e-3), ("fp32", 1.5e-6)):
        q, k, v = inputs(T, 1, 1, D, dtype, 31)
        s = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        got = xq.prompt_attn(q, k, v, s)[-40:, 0]
        z = (q[-40:, 0].double() @ k[:, 0].double().T) * D ** -0.5
        at = torch.arange(T, device="cuda")
        z = z.masked_fill(at > at[-40:, None], -math.inf)
        assert ops_check.rms(got, torch.softmax(z, -1) @ v[:, 0].double()) <= limit
