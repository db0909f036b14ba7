"""Low-rank adapters beside projections, against 64 bits."""
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


def adapters(n, rank, K, N, dtype, seed=0, scaled=True):
    g = torch.Generator("cuda").manual_seed(seed)
    a = (torch.randn(n, rank, K, device="cuda", generator=g) * K ** -0.5).to(DTYPES[dtype])
    b = (torch.randn(n, N, rank, device="cuda", generator=g) * rank ** -0.5).to(DTYPES[dtype])
    return a, b, torch.rand(n, device="cuda", generator=g) * 2 - 1 if scaled else None


def run(xq, M, projs, ids, seed=1):
    """projs: ((a, b, scales), K) tuples, each with an input of its own width."""
    g = torch.Generator("cuda").manual_seed(seed)
    widths = sorted({p[0].shape[2] for p in projs})
    inputs = [torch.randn(M, k, device="cuda", generator=g) for k in widths]
    at = [widths.index(p[0].shape[2]) for p in projs]
    ys = [torch.randn(M, p[1].shape[1], device="cuda", generator=g) for p in projs]
    before = [y.clone() for y in ys]
    got = xq.Adapters([(*p, i) for p, i in zip(projs, at)]).add(inputs, ys, ids)
    torch.cuda.synchronize()
    for p, i, y, y0 in zip(projs, at, got, before):
        want, bound = ops_check.lora(inputs[i], *p, ids, y0)
        ops_check.within(y, want, bound)
        none = (ids < 0) | (ids >= p[0].shape[0])
        assert torch.equal(y[none], y0[none])
    return inputs, before, got


def some_ids(M, n, seed=3, spread="mixed", idle=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1 if idle else 0, n, (M,), generator=g, dtype=torch.int32)
    return (ids if spread == "mixed" else ids.sort().values).cuda()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,n,rank,K,N", [
    (1, 1, 8, 32, 1), (1, 3, 16, 4096, 4096), (2, 2, 24, 96, 77), (7, 4, 64, 512, 130), (8, 40, 16, 1536, 256), (33, 5, 128, 256, 1000),
    (64, 64, 8, 1024, 515), (65, 3, 32, 4096, 1024), (129, 2, 256, 288, 192), (257, 7, 40, 1536, 1536), (1000, 4, 16, 512, 2048),
    (515, 300, 8, 64, 33)])
@pytest.mark.parametrize("spread", ["mixed", "packed"])
def test_rows_get_their_adapters(xq, dtype, M, n, rank, K, N, spread):
    run(xq, M, [adapters(n, rank, K, N, dtype)], some_ids(M, n, spread=spread))


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,n,rank,K,N", [
    (1, 1, 256, 32, 4100), (4, 2, 128, 4096, 9001), (16, 1, 64, 544, 4096), (16, 1, 72, 512, 300), (17, 1, 136, 1056, 130), (90, 2, 40, 2048, 515),
    (33, 5, 248, 96, 77), (2431, 30, 16, 64, 36), (2432, 30, 16, 64, 36), (2500, 9, 64, 512, 264), (2450, 3, 256, 96, 130), (2600, 40, 8, 32, 77),
])
def test_ranks_and_rows_shared_out_otherwise(xq, dtype, M, n, rank, K, N):
    run(xq, M, [adapters(n, rank, K, N, dtype)], some_ids(M, n, idle=M > 16))


@pytest.mark.parametrize("M", [1, 5, 64, 300])
def test_projections_together(xq, M):
    """Widths, ranks, types and numbers of adapters that differ, two inputs, one projection without scales."""
    projs = [adapters(6, 16, 1536, 1536, "bf16", 1), adapters(6, 8, 1536, 256, "fp16", 2, scaled=False), adapters(9, 64, 1536, 77, "fp32", 3),
             adapters(6, 32, 8960, 1536, "bf16", 4)]
    run(xq, M, projs, some_ids(M, 6))


def test_ids_that_no_adapter_has(xq):
    """Too large ones are left out and recorded, and none of the rest suffers."""
    assert xq.device_error() == 0
    ids = torch.tensor([0, 5, 2, -7, 2147483647, 1, -2147483648, 3] * 20, dtype=torch.int32, device="cuda")
    run(xq, 160, [adapters(3, 16, 512, 256, "bf16")], ids)
    assert xq.device_error() == 5 << 8 | 1
    assert xq.device_error() == 0
    # a projection may have fewer adapters than another
    run(xq, 8, [adapters(4, 16, 512, 256, "bf16"), adapters(1, 16, 512, 64, "bf16")], ids[:8].clamp(-1, 3))
    assert xq.device_error() == 5 << 8 | 1


def test_no_rows_no_adapters_no_columns(xq):
    a, b, s = adapters(3, 16, 512, 64, "bf16")
    xq.Adapters([(a, b, s, 0)]).add([torch.zeros(0, 512, device="cuda")], [torch.zeros(0, 64, device="cuda")],
                                    torch.zeros(0, dtype=torch.int32, device="cuda"))
    run(xq, 9, [(a, b, s)], torch.full((9,), -1, dtype=torch.int32, device="cuda"))
    run(xq, 9, [(a[:0], b[:0], s[:0])], torch.full((9,), -1, dtype=torch.int32, device="cuda"))
    run(xq, 9, [(a, b[:, :0].contiguous(), s), (a, b, s)], some_ids(9, 3))
    assert xq.device_error() == 0


@pytest.mark.parametrize("M", [3, 200])
def test_rows_are_apart(xq, M):
    """A row's result does not depend on other rows' values, not on infinities or NaN either; nor do adapters on each other."""
    a, b, s = adapters(4, 16, 512, 192, "bf16")
    ids = some_ids(M, 3, idle=False)
    ids[0] = 3
    inputs, before, got = run(xq, M, [(a, b, s)], ids)
    x, y = inputs[0].clone(), before[0].clone()
    x[0], y[0] = float("nan"), 0
    x[0, ::2] = float("inf")
    a2, b2 = a.clone(), b.clone()
    a2[3], b2[3] = float("inf"), float("nan")
    xq.Adapters([(a2, b2, s, 0)]).add([x], [y], ids)
    assert torch.equal(y[1:], got[0][1:]) and bool(torch.isnan(y[0]).all())


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_sizes_far_apart(xq, dtype):
    """x of 2^60 and 2^-60 and adapters down to the type's subnormal numbers: products keep fp32's precision."""
    a, b, s = adapters(2, 16, 256, 64, dtype)
    a, b = a * 2.0 ** -13, b * 2.0 ** -13
    ids = some_ids(40, 2, idle=False)
    for power in (60, -60):
        x = torch.randn(40, 256, device="cuda") * 2.0 ** power
        y = torch.zeros(40, 64, device="cuda")
        want, bound = ops_check.lora(x, a, b, s, ids, y)
        xq.Adapters([(a, b, s, 0)]).add([x], [y], ids)
        ops_check.within(y, want, bound)


@pytest.mark.parametrize("M,spread", [(5, "mixed"), (64, "mixed"), (700, "packed"), (700, "mixed")])
def test_root_mean_square(xq, M, spread):
    """As near to 64 bits as fp32 operations are: errors that add up at random, some sqrt(K) steps of 2^-24."""
    a, b, s = adapters(6, 32, 4096, 512, "bf16", scaled=False)
    ids = some_ids(M, 6, spread=spread, idle=False)
    x, y = torch.randn(M, 4096, device="cuda"), torch.zeros(M, 512, device="cuda")
    want, _ = ops_check.lora(x, a, b, s, ids, y)
    xq.Adapters([(a, b, s, 0)]).add([x], [y], ids)
    assert ops_check.rms(y, want) <= 64 * 2.0 ** -24 / 4


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,n,rank,K,N", [(5, 4, 128, 8960, 1536), (3, 1, 256, 512, 4096), (3000, 4, 128, 4096, 1536), (3000, 2, 256, 1024, 520)])
def test_sums_over_ranks_do_not_drift(xq, dtype, M, n, rank, K, N):
    """A cut-off addition loses 2^-24 of the running sum on average and 2^-23 at most, always towards 0: with up to six between
    two sums in fp32 that is 6 x 2^-24 of a product, 12 x 2^-24 for both; the dropped products of two lower halves are another
    2^-22 / 4 each, and fp32 roundings at random some 3 x 2^-24: 17 x 2^-24 in all."""
    a, b, s = adapters(n, rank, K, N, dtype, scaled=False)
    ids = some_ids(M, n, idle=False)
    x, y = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(9)), torch.zeros(M, N, device="cuda")
    want, _ = ops_check.lora(x, a, b, s, ids, y)
    xq.Adapters([(a, b, s, 0)]).add([x], [y], ids)
    assert ops_check.rms(y, want) <= 17 * 2.0 ** -24


def test_repeated_captured_and_on_another_stream(xq):
    """Bit for bit the same: no result depends on timing."""
    a, b, s = adapters(5, 16, 1024, 300, "fp16")
    for M in (1, 37, 400):
        ids = some_ids(M, 5)
        x, y0 = torch.randn(M, 1024, device="cuda"), torch.randn(M, 300, device="cuda")
        ad = xq.Adapters([(a, b, s, 0)])
        want = ad.add([x], [y0.clone()], ids)[0]
        for _ in range(5):
            assert torch.equal(ad.add([x], [y0.clone()], ids)[0], want)
        side, y = torch.cuda.Stream(), y0.clone()
        side.wait_stream(torch.cuda.current_stream())
        ad.add([x], [y], ids, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, want)
        g = torch.cuda.CUDAGraph()
        y = y0.clone()
        with torch.cuda.graph(g):
            ad.add([x], [y], ids)
        assert torch.equal(y, y0)
        g.replay()
        assert torch.equal(y, want)
        ids.fill_(-1)  # a replay goes by what the ids hold then
        g.replay()
        assert torch.equal(y, want)


def test_a_layer_with_adapters(xq):
    from gguf_quant_integer_gb300 import synth
    projs = (synth.Proj("q", synth.Q4_K, 512, 256, 0), synth.Proj("v", synth.Q6_K, 512, 130, 0), synth.Proj("down", synth.Q6_K, 768, 512, 1))
    ws = [synth.gen_weight(p.qtype, 40 + t, p.N, p.K) for t, p in enumerate(projs)]
    ad = {0: adapters(3, 16, 512, 256, "bf16"), 2: adapters(3, 8, 768, 512, "fp16")}
    for M in (2, 20, 100):
        layer = xq.Layer(projs, ws, M, adapters=ad)
        inputs = [torch.randn(M, 512, device="cuda"), torch.randn(M, 768, device="cuda")]
        plain = [y.clone() for y in layer.forward(inputs)]
        ids = some_ids(M, 3)
        got = layer.forward(inputs, ids=ids)
        torch.cuda.synchronize()
        assert torch.equal(got[1], plain[1])
        for i, x in ((0, inputs[0]), (2, inputs[1])):
            want, bound = ops_check.lora(x, *ad[i], ids, plain[i])
            ops_check.within(got[i], want, bound)
    with pytest.raises(ValueError):
        xq.Layer(projs, ws, 2).forward([x[:2] for x in inputs], ids=ids[:2])
    with pytest.raises(ValueError):
        xq.Layer(projs, ws, 2, adapters={1: ad[0]})


def test_refusals(xq):
    a, b, s = adapters(3, 16, 512, 64, "bf16")
    x, y, ids = torch.zeros(4, 512, device="cuda"), torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ([], [(a, b, s, -1)], [(a[0], b, s, 0)], [(a, b.half(), s, 0)], [(a, b, s[:2], 0)], [(a, b, s.double(), 0)],
                [(a[:, :12].contiguous(), b[:, :, :12].contiguous(), s, 0)], [(a[:, :, :40].contiguous(), b, s, 0)],
                [(a.transpose(1, 2), b, s, 0)], [(a.cpu(), b, s, 0)], [(a.double(), b.double(), s, 0)], [(a, b, s, 0)] * 17):
        with pytest.raises(ValueError):
            xq.Adapters(bad)
    ad = xq.Adapters([(a, b, s, 0)])
    for args in (([x], [y], ids.long()), ([x], [y], ids[::2]), ([x[:3]], [y], ids), ([x], [y[:, :63]], ids), ([x], [], ids), ([], [y], ids),
                 ([x.half()], [y], ids), ([x], [y.half()], ids), ([x.cpu()], [y], ids), ([x], [y], ids.cpu()),
                 ([torch.zeros(4, 1024, device="cuda")[:, :512]], [y], ids)):
        with pytest.raises(ValueError):
            ad.add(*args)
    with pytest.raises(xq.XQError):  # not on a 16-byte boundary
        ad.add([torch.zeros(4 * 512 + 1, device="cuda")[1:].view(4, 512)], [y], ids)
