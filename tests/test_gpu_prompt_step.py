"""Adapters, norms with rotation, prompt attention and the cache as a program uses them: packed prompts of requests with
adapters of their own through a layer's attention half, then one token of each."""
import math

import pytest
import torch

import ops_check
from gguf_quant_integer_gb300 import build as xqbuild, synth

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 512, 8, 2, 64, 16
LENS = (40, 1, 131)  # of the prompts


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    return _xq


def adapters(rank, K, N, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return ((torch.randn(2, rank, K, device="cuda", generator=g) * K ** -0.5).bfloat16(),
            (torch.randn(2, N, rank, device="cuda", generator=g) * rank ** -0.5).bfloat16(), torch.rand(2, device="cuda", generator=g))


class Half:
    """q, k and v projections with adapters beside q and v, norms and rotation, attention, cache."""

    def __init__(self, xq, M):
        self.xq, kv = xq, KV_HEADS * DIM
        projs = (synth.Proj("q", synth.Q4_K, HIDDEN, HEADS * DIM, 0), synth.Proj("k", synth.Q4_K, HIDDEN, kv, 0),
                 synth.Proj("v", synth.Q6_K, HIDDEN, kv, 0))
        self.ad = {0: adapters(16, HIDDEN, HEADS * DIM, 1), 2: adapters(8, HIDDEN, kv, 2)}
        self.layer = xq.Layer(projs, [synth.gen_weight(p.qtype, i, p.N, p.K) for i, p in enumerate(projs)], M, adapters=self.ad)
        g = torch.Generator("cuda").manual_seed(3)
        self.qw, self.kw = (1 + 0.2 * torch.randn(DIM, device="cuda", generator=g) for _ in range(2))
        self.rope = xq.Rope(DIM, base=1e4)

    def qkv(self, x, ids, positions, dtype=None):
        q, k, v = self.layer.forward([x], ids=ids)
        q, k = self.xq.qk_norm_rope(q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), positions, self.rope, self.qw, self.kw, dtype=dtype)
        return q, k, v.unflatten(1, (KV_HEADS, DIM))


def test_prompts_then_a_token(xq):
    starts = [0]
    for n in LENS:
        starts.append(starts[-1] + n)
    T, B = starts[-1], len(LENS)
    g = torch.Generator("cuda").manual_seed(7)
    x, x1 = (torch.randn(n, HIDDEN, device="cuda", generator=g) * 0.1 for n in (T, B))
    request = torch.tensor([0, -1, 1], dtype=torch.int32, device="cuda")  # adapters; the second request has none
    lens = torch.tensor(LENS, device="cuda")
    owner = torch.repeat_interleave(torch.arange(B, device="cuda"), lens)
    first = torch.tensor(starts, dtype=torch.int32, device="cuda")
    positions = torch.arange(T, device="cuda") - first[:-1].long()[owner]

    whole = Half(xq, T)
    q, k, v = whole.qkv(x, request[owner].contiguous(), positions)
    out = xq.prompt_attn(q, k, v, first)
    torch.cuda.synchronize()
    assert xq.device_error() == 0
    # the projections' adapters
    plain = [y.clone() for y in whole.layer.forward([x])]
    for i in (0, 2):
        want, bound = ops_check.lora(x, *whole.ad[i], request[owner], plain[i])
        ops_check.within(whole.layer.forward([x], ids=request[owner].contiguous())[i], want, bound)
    # norms, rotation and attention
    plain = whole.layer.forward([x], ids=request[owner].contiguous())
    want, bound = ops_check.norm_rope(plain[0].unflatten(1, (HEADS, DIM)), positions, 1e4, DIM, False, whole.qw, 1e-6, torch.float32)
    ops_check.within(q, want, bound)
    want, bound = ops_check.attention(q, k, v, starts, DIM ** -0.5)
    ops_check.within(out, want, bound)

    # the prompts into the cache, then one token of each request: the cache's attention is the prompt's over one token more,
    # but for the blocks' rounding (Q8_0: half a step of a 127th of a block's largest)
    step = Half(xq, B)
    q1, k1, v1 = step.qkv(x1, request, lens)
    pages = [-(-(n + 1) // PAGE) for n in LENS]
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :pages[b]] = torch.arange(sum(pages[:b]), sum(pages[:b + 1]))
    table = table.cuda()
    cache = xq.KVCache(xq.XQ_TYPE_Q8_0, sum(pages), PAGE, KV_HEADS, DIM)
    slot = lambda b, t: table[b, t // PAGE].long() * PAGE + t % PAGE  # noqa: E731
    cache.write(k, v, slot(owner, positions))
    cache.write(k1, v1, slot(torch.arange(B, device="cuda"), lens))
    got = cache.attn(q1.unsqueeze(1), table, (lens + 1).int())[:, 0]
    parts = []  # the prompts with the token behind each
    for a, a1 in ((q, q1), (k, k1), (v, v1)):
        parts.append(torch.cat([t for b in range(B) for t in (a[starts[b]:starts[b + 1]], a1[b:b + 1])]))
    more = torch.tensor([s + b for b, s in enumerate(starts)], dtype=torch.int32, device="cuda")
    want = xq.prompt_attn(*parts, more)[(more[1:] - 1).long()]
    assert ops_check.rms(got, want.double()) <= 0.02
    # and exactly so over what the cache holds
    kc, vc = (torch.cat([z[starts[b] + b:starts[b + 1] + b + 1] for b in range(B)]) for z in (
        t for t in cache.read(torch.cat([slot(torch.full((n + 1,), b, device="cuda"), torch.arange(n + 1, device="cuda")) for b, n in enumerate(LENS)]))))
    want = xq.prompt_attn(parts[0], kc, vc, more)[(more[1:] - 1).long()]
    assert ops_check.rms(got, want.double()) <= 3e-6
    assert xq.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_16_bit_prompts(xq, dtype):
    """Norms and rotation hand over what 16-bit attention reads; all in one captured graph, run again on other inputs."""
    T, starts = 172, torch.tensor([0, 40, 41, 172], dtype=torch.int32, device="cuda")
    half = Half(xq, T)
    x, ids = torch.randn(T, HIDDEN, device="cuda") * 0.1, (torch.arange(T, device="cuda") % 3 - 1).int()
    positions = torch.arange(T, device="cuda")

    def run():
        q, k, v = half.qkv(x, ids, positions, dtype)
        return q, k, v.to(dtype), xq.prompt_attn(q, k, v.to(dtype), starts)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = run()
    x.copy_(torch.randn(T, HIDDEN, device="cuda") * 0.1)
    g.replay()
    again = run()
    torch.cuda.synchronize()
    for a, b in zip(captured, again):
        assert torch.equal(a, b)
    want, bound = ops_check.attention(*again[:3], starts.tolist(), DIM ** -0.5)
    ops_check.within(again[3], want, bound)
    assert math.isfinite(float(again[3].float().sum()))
