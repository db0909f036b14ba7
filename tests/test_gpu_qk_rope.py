"""Norms of queries and keys with the position rotation, against 64 bits."""
import pytest
import torch

import ops_check
from gguf_quant_integer_gb300 import build as xqbuild
from ops_check import DTYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    return _xq


def case(xq, T=5, H=4, Hk=2, D=128, rot=128, pairs=False, dtype="fp32", out="fp32", norm=True, base=1e6, positions=None, fused=False,
         lead=0, eps=1e-6, magnitude=1.0, factors=None, seed=0, x=None):
    g = torch.Generator("cuda").manual_seed(seed)
    row = (H + 2 * Hk) * D + lead
    x = (torch.randn(T, row, device="cuda", generator=g) if x is None else x).to(DTYPES[dtype])
    q, k = x[:, lead:lead + H * D], x[:, lead + H * D:lead + (H + Hk) * D]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    q, k = q.unflatten(1, (H, D)), k.unflatten(1, (Hk, D))
    qw, kw = (1 + 0.5 * torch.randn(D, device="cuda", generator=g) for _ in range(2)) if norm else (None, None)
    positions = torch.arange(T, device="cuda") if positions is None else torch.tensor(positions, device="cuda")
    before = x.clone()
    rope = xq.Rope(rot, base, factors, pairs, magnitude)
    got = xq.qk_norm_rope(q, k, positions, rope, qw, kw, eps=eps, dtype=DTYPES[out])
    torch.cuda.synchronize()
    for y, z, w in zip(got, (q, k), (qw, kw)):
        want, bound = ops_check.norm_rope(z, positions, base, rot, pairs, w, eps, DTYPES[out], magnitude, factors)
        assert y.dtype == DTYPES[out] and y.is_contiguous()
        ops_check.within(y, want, bound)
    assert torch.equal(x, before)
    return q, k, positions, rope, qw, kw, got


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,H,Hk,D,rot,pairs", [
    (1, 32, 8, 128, 128, False), (3, 12, 2, 128, 128, True), (257, 5, 1, 64, 64, False), (33, 16, 16, 96, 96, False),
    (33, 3, 1, 96, 48, True), (7, 16, 2, 256, 256, False), (7, 1, 1, 256, 64, True), (40, 7, 7, 64, 32, False), (3, 9, 4, 128, 16, False),
    (2, 2, 1, 128, 0, False), (1000, 32, 8, 128, 64, False)])
def test_rows_are_normalized_and_turned(xq, dtype, out, T, H, Hk, D, rot, pairs):
    case(xq, T, H, Hk, D, rot, pairs, dtype, out, norm=T % 2 == 1)


@pytest.mark.parametrize("pairs", [False, True])
def test_far_and_negative_positions(xq, pairs):
    """The oracle's own angles, products in 64 bits, carry 2^-52 of the position: their bound grows, the kernel's does not."""
    case(xq, 8, positions=[0, 1, -1, 131071, 1 << 20, -(1 << 31), (1 << 24) + 1, 99999999], pairs=pairs, norm=False)


def test_positions_past_32_bits(xq):
    """Angles of 2^40 + p and p differ by those of 2^40: turning by one after the other is turning by both."""
    q, k, pos, rope, *_ = case(xq, 6, norm=False, positions=[0, 1, 5, 17, 1000, 12345])
    far = pos + (1 << 40)
    both, _ = xq.qk_norm_rope(q, k, far, rope)
    first, fk = xq.qk_norm_rope(q, k, torch.full_like(pos, 1 << 40), rope)
    again, _ = xq.qk_norm_rope(first, fk, pos, rope)
    assert float((both - again).abs().max()) <= 12 * 2.0 ** -24 * float(q.abs().max()) * 2


def test_angles_are_whole_number_arithmetic(xq):
    """Equal rows at positions a full turn apart get equal bits (a table whose turns are exact)."""
    rope = xq.Rope(128)
    rope.turns.fill_(1 << 60)  # a sixteenth of a turn
    x = torch.randn(1, 4, 128, device="cuda").expand(3, 4, 128).contiguous()
    q, k = xq.qk_norm_rope(x, x[:, :2].contiguous(), torch.tensor([3, 3 + 16, 3 - 160000000], device="cuda"), rope)
    assert torch.equal(q[0], q[1]) and torch.equal(q[0], q[2])


@pytest.mark.parametrize("lead", [0, 8, 3])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_views_of_a_longer_row(xq, lead, dtype):
    """Rows on and off 16-byte boundaries."""
    case(xq, 9, 12, 2, 128, fused=True, lead=lead, dtype=dtype, out=dtype)
    case(xq, 9, 3, 1, 96, 96, fused=True, lead=lead, dtype=dtype, out="fp16")


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_in_place(xq, dtype):
    q, k, pos, rope, qw, kw, want = case(xq, 70, 6, 3, 96, 96, dtype=dtype, out=dtype, fused=True)
    got = xq.qk_norm_rope(q, k, pos, rope, qw, kw, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_factors_magnitude_and_eps(xq):
    g = torch.Generator().manual_seed(0)
    case(xq, 20, factors=1 + 7 * torch.rand(64, generator=g), magnitude=1.25, eps=0.5)
    case(xq, 20, rot=64, pairs=True, magnitude=-0.5, norm=False, base=1e4)
    case(xq, 20, eps=0.0)


def test_rows_of_zeros_and_rows_far_from_one(xq):
    x = torch.randn(6, 8 * 128, device="cuda") * torch.tensor([1.0, 0.0, 2.0 ** 50, 2.0 ** -50, 2.0 ** -100, 1.0], device="cuda")[:, None]
    case(xq, 4, x=x[:4].contiguous())
    case(xq, 6, x=x, norm=False)


def test_what_is_not_finite_stays_in_its_row(xq):
    """Without norms it stays in its pair, and rows beside it are as without it."""
    q, k, pos, rope, qw, kw, want = case(xq, 5, rot=64)
    bad = q.clone()
    bad[2, 1, 3] = float("inf")
    got, gk = xq.qk_norm_rope(bad, k, pos, rope, qw, kw)
    keep = torch.ones(5, 4, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(got[keep], want[0][keep]) and torch.equal(gk, want[1])
    plain, _ = xq.qk_norm_rope(q, k, pos, rope)
    got, _ = xq.qk_norm_rope(bad, k, pos, rope)
    same = torch.ones(5, 4, 128, dtype=torch.bool)
    same[2, 1, 3] = same[2, 1, 3 + 32] = False
    assert torch.equal(got[same], plain[same]) and not bool(torch.isfinite(got[2, 1, 3]))
    bad = q.clone()
    bad[2, 1, 100] = float("nan")  # not among the turned ones
    got, _ = xq.qk_norm_rope(bad, k, pos, rope)
    same = torch.ones(5, 4, 128, dtype=torch.bool)
    same[2, 1, 100] = False
    assert torch.equal(got[same], plain[same]) and bool(torch.isnan(got[2, 1, 100]))


def test_streams_and_graphs(xq):
    q, k, pos, rope, qw, kw, want = case(xq, 33)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = xq.qk_norm_rope(q, k, pos, rope, qw, kw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = xq.qk_norm_rope(q, k, pos, rope, qw, kw)
    pos += 5
    g.replay()
    c, d = xq.qk_norm_rope(q, k, pos, rope, qw, kw)
    assert torch.equal(a, c) and torch.equal(b, d) and not torch.equal(a, want[0])


def test_refusals_and_empty_calls(xq):
    q, k = torch.zeros(4, 4, 128, device="cuda"), torch.zeros(4, 2, 128, device="cuda")
    pos, rope, w = torch.arange(4, device="cuda"), xq.Rope(128), torch.ones(128, device="cuda")
    ok = dict(q=q, k=k, positions=pos, rope=rope)
    for kw in (dict(k=k[:3]), dict(k=k.half()), dict(k=k.cpu()), dict(positions=pos.int()), dict(positions=pos[:3]), dict(positions=pos.cpu()),
               dict(q_weight=w[:64]), dict(q_weight=w.half()), dict(k_weight=w.cpu()), dict(q=q.double(), k=k.double()),
               dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q_out=q.half(), dtype=q.dtype), dict(k_out=k[:, :, :64]),
               dict(dtype=torch.float64), dict(rope=xq.Rope(128, device="cpu"))):
        with pytest.raises(ValueError):
            xq.qk_norm_rope(**{**ok, **kw})
    for kw in (dict(rope=xq.Rope(256)), dict(eps=-1.0), dict(eps=float("nan")), dict(q=q[:, :, :32].contiguous(), k=k[:, :, :32].contiguous())):
        with pytest.raises(xq.XQError):
            xq.qk_norm_rope(**{**ok, **kw})
    with pytest.raises(ValueError):
        xq.Rope(24)
    with pytest.raises(ValueError):
        xq.Rope(32, factors=[1.0] * 15)
    with pytest.raises(ValueError):
        xq.Rope(32, factors=[0.0] * 16)
    a, b = xq.qk_norm_rope(q[:0], k[:0], pos[:0], rope)
    assert a.shape == (0, 4, 128) and b.shape == (0, 2, 128)
    one, _ = xq.qk_norm_rope(q[:1].expand(1, 4, 128), k[:1], pos[:1], rope)
    assert one.shape == (1, 4, 128)
