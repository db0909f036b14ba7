#!/usr/bin/env python
"""One decode step of a layer's attention half, from quantized weights to quantized weights.

A batch of sequences continues one shared prompt. The step runs what an engine
would: q, k and v projections from GGUF weights (xq_layer_mixed), norms of q and
k for each head with the position rotation (xq_qk_norm_rope), the new K and
V rows into the paged cache (xq_kv_write), attention over the shared prompt and
each sequence's own tokens (xq_kv_attn_shared), and the output projection. The
cached rows of the prompt and of the first new tokens are written the same way
beforehand, and read back at the end (xq_kv_read) to check the attention in 64
bits.

    python examples/decode_step.py [--batch 8] [--prompt 1000] [--steps 4] [--cache q8_0|q4_0]
"""
import argparse
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from gguf_quant_integer_gb300 import build, synth, xq  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1536, 12, 2, 128, 64


class AttentionHalf:
    """The layer's weights, its cache, and the page tables of a batch that shares a prompt."""

    def __init__(self, batch, prompt, most, cache_type, seed=0):
        import torch
        self.torch, self.batch, self.prompt = torch, batch, prompt
        kv = KV_HEADS * DIM
        self.qkv = [synth.Proj("q", synth.Q4_K, HIDDEN, HEADS * DIM, 0), synth.Proj("k", synth.Q4_K, HIDDEN, kv, 0),
                    synth.Proj("v", synth.Q6_K, HIDDEN, kv, 0)]
        self.o = [synth.Proj("o", synth.Q4_K, HEADS * DIM, HIDDEN, 0)]
        self.w = [synth.gen_weight(p.qtype, seed + i, p.N, p.K) for i, p in enumerate(self.qkv + self.o)]
        self.layer = xq.Layer(self.qkv, self.w[:3], batch)
        self.out = xq.Layer(self.o, self.w[3:], batch)
        # pages: the prompt's, then `own` of each sequence, handed out in a scattered order
        head, own = -(-prompt // PAGE), -(-most // PAGE)
        order = torch.from_numpy(np.random.default_rng(seed).permutation(head + batch * own).astype(np.int32)).cuda()
        self.cache = xq.KVCache(cache_type, head + batch * own, PAGE, KV_HEADS, DIM)
        self.prompt_pages, self.pages = order[:head].contiguous(), order[head:].view(batch, own).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        gen = torch.Generator("cuda").manual_seed(seed)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(DIM, device="cuda", generator=gen) for _ in range(2))
        self.rope = xq.Rope(DIM, base=1e6)

    def turned(self, q, k, positions):
        """q and k rows normalized for each head and rotated to their positions, in place."""
        q, k = q.view(-1, HEADS, DIM), k.view(-1, KV_HEADS, DIM)
        return xq.qk_norm_rope(q, k, positions, self.rope, self.q_norm, self.k_norm, q_out=q, k_out=k)

    def prefill(self, x):
        """K and V of the prompt's inputs x [prompt, HIDDEN] into its pages; the prompt's own attention."""
        torch = self.torch
        a = xq.quantize_q8(x)
        q, k, v = (xq.matmul(p.qtype, self.layer.W[i], a, self.prompt, p.N, p.K) for i, p in enumerate(self.qkv))
        t = torch.arange(self.prompt, device="cuda")
        q, k = self.turned(q, k, t)
        self.prompt_slots = self.prompt_pages[t // PAGE].long() * PAGE + t % PAGE
        self.cache.write(k.view(-1, KV_HEADS, DIM), v.view(-1, KV_HEADS, DIM), self.prompt_slots)
        starts = torch.tensor([0, self.prompt], dtype=torch.int32, device="cuda")
        return xq.prompt_attn(q, k, v.view(-1, KV_HEADS, DIM), starts)

    def step(self, x):
        """One token of each sequence: x [batch, HIDDEN] -> the half's output [batch, HIDDEN]."""
        torch = self.torch
        q, k, v = self.layer.forward([x])
        at = self.lens.long()
        q, k = self.turned(q, k, self.prompt + at)
        slots = self.pages.gather(1, (at // PAGE)[:, None])[:, 0].long() * PAGE + at % PAGE
        self.cache.write(k.view(-1, KV_HEADS, DIM), v.view(-1, KV_HEADS, DIM), slots)
        self.lens += 1
        self.q = q.view(self.batch, 1, HEADS, DIM)
        self.attended = self.cache.attn_shared(self.q, self.prompt_pages, self.prompt, self.pages, self.lens)
        y, = self.out.forward([self.attended.view(self.batch, HEADS * DIM)])
        torch.cuda.current_stream().synchronize()
        return y

    def error(self):
        """Largest error of the last step's attention against 64 bits, over its largest value."""
        torch = self.torch
        worst = 0.0
        pk, pv = (t.double() for t in self.cache.read(self.prompt_slots))
        for b in range(self.batch):
            t = torch.arange(int(self.lens[b]), device="cuda")
            own = self.pages[b][t // PAGE].long() * PAGE + t % PAGE
            k, v = (torch.cat((p, o.double())) for p, o in zip((pk, pv), self.cache.read(own)))
            q = self.q[b, 0].double().view(KV_HEADS, -1, DIM)
            w = torch.softmax(torch.einsum("hgd,lhd->hgl", q, k) * DIM ** -0.5, -1)
            want = torch.einsum("hgl,lhd->hgd", w, v).reshape(HEADS, DIM)
            worst = max(worst, float((self.attended[b, 0].double() - want).abs().max() / want.abs().max()))
        return worst


def main(argv=None):
    import torch
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--cache", choices=("q8_0", "q4_0"), default="q8_0")
    a = p.parse_args(argv)
    build.build()
    half = AttentionHalf(a.batch, a.prompt, a.steps, xq.XQ_TYPE_Q8_0 if a.cache == "q8_0" else xq.XQ_TYPE_Q4_0)
    # the weights are random, so inputs are scaled to give scores of ordinary size
    make = lambda seed, n: torch.from_numpy(synth.gen_x(seed, n, HIDDEN) * np.float32(0.02)).cuda()  # noqa: E731
    half.prefill(make(100, a.prompt))
    for i in range(a.steps):
        y = half.step(make(200 + i, a.batch))
    err, bad = half.error(), xq.device_error()
    print(f"{a.steps} steps, {a.batch} sequences after a prompt of {a.prompt}, cache {a.cache} of {half.cache.k.numel() * 2} bytes: "
          f"output {tuple(y.shape)}, attention within {err:.1e} of 64 bits, device record {bad}")
    if not torch.isfinite(y).all() or err > 1e-5 or bad:
        raise SystemExit("the step's results are off")
    return y


if __name__ == "__main__":
    main()
