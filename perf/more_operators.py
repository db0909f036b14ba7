"""Timed cases of what stands between a layer's quantized projections and its KV cache.

Three operators, in the order in which a prompt or a decode step meets them:

  lora    low-rank adapters of many requests beside projections that share an input: each row of x goes through
          the adapter that its id names (none where it is negative), y += scale * (x A^T) B^T
  rope    norms of queries and keys for each head, with the position rotation in the same pass
  attn    causal attention over whole prompts with grouped heads, packed one behind the other

`own` selects what run() calls: this package's kernels, or the same mathematics as elementary torch
operations in fp32.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
# Query heads, KV heads and head size of an attention layer: the 8B-class layer (4096 and 1024 wide q and k/v projections),
# the 1.5B-class one (1536 and 256 wide), and generic ones with other groupings and head sizes.
HEADS = ((32, 8, 128), (12, 2, 128), (8, 8, 64), (14, 2, 64), (16, 16, 96), (21, 3, 128), (16, 2, 256), (5, 1, 64))
# Input width and output widths of projections that share an input: 8B-class q/k/v, gate/up and o, 1.5B-class q/k/v, gate/up
# and down, a 14B-class ffn, a small one of odd width.
WIDTHS = ((4096, (4096, 1024, 1024)), (4096, (14336, 14336)), (4096, (4096,)), (1536, (1536, 256, 256)), (1536, (8960, 8960)),
          (8960, (1536,)), (5120, (17408,)), (512, (130, 77)))
EPS = 1e-6


def listed():
    return [
        # One request's decode step at one projection: a call of almost no work.
        dict(name="lora_token_bf16", op="lora", dtype="bf16", tokens=1, spread="packed", requests=1, adapters=4, idle=0, rank=16, width=2),
        # A decode step of 64 requests over 16 adapters out of a store of 40, at q, k and v together.
        dict(name="lora_decode_bf16", op="lora", dtype="bf16", tokens=64, spread="mixed", requests=16, adapters=40, idle=0, rank=16, width=0),
        # Rows of decode and prompt steps mixed in one call, fp16 adapters, one row in five without one.
        dict(name="lora_mixed_fp16", op="lora", dtype="fp16", tokens=777, spread="mixed", requests=9, adapters=9, idle=5, rank=8, width=4),
        # Prompts of several requests behind each other, at the widest projections.
        dict(name="lora_prompt_bf16", op="lora", dtype="bf16", tokens=4099, spread="packed", requests=6, adapters=8, idle=0, rank=64, width=1),
        # One new token of one sequence, in the fp32 that the projections give.
        dict(name="rope_token_fp32", op="rope", dtype="fp32", out="fp32", tokens=1, hq=32, heads=8, dim=128, rot=128, fused=0, norm=1,
             pairs=0, base=1e6, start=131071),
        # A wide decode batch: q and k are views of one row, rotated in neighbouring pairs, without norms.
        dict(name="rope_batch_bf16", op="rope", dtype="bf16", out="bf16", tokens=257, hq=12, heads=2, dim=128, rot=128, fused=1, norm=0,
             pairs=1, base=1e4, start=0),
        # A long prompt's part at far positions, from the projections' fp32 into what the attention reads.
        dict(name="rope_prompt_fp32_bf16", op="rope", dtype="fp32", out="bf16", tokens=16383, hq=32, heads=8, dim=128, rot=128, fused=0,
             norm=1, pairs=0, base=1e6, start=100000),
        # A short question alone: latency is all.
        dict(name="attn_short_bf16", op="attn", dtype="bf16", batch=1, hq=32, heads=8, dim=128, lo=97, hi=97, fused=0, window=0),
        # Prompts of all lengths packed into one call, q, k and v as views of one row.
        dict(name="attn_packed_bf16", op="attn", dtype="bf16", batch=16, hq=32, heads=8, dim=128, lo=17, hi=2048, fused=1, window=0),
        # One long document.
        dict(name="attn_long_bf16", op="attn", dtype="bf16", batch=1, hq=32, heads=8, dim=128, lo=12287, hi=12287, fused=0, window=0),
        # A few documents under a sliding window, 1.5B-class heads.
        dict(name="attn_window_fp16", op="attn", dtype="fp16", batch=4, hq=12, heads=2, dim=128, lo=300, hi=4099, fused=0, window=1024),
        # Prompts in the fp32 that the projections give.
        dict(name="attn_packed_fp32", op="attn", dtype="fp32", batch=5, hq=32, heads=8, dim=128, lo=33, hi=1500, fused=0, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("lora", "lora", "rope", "attn", "attn"))
    dtype = rng.choice(("fp32", "fp16", "bf16"))
    hq, heads, dim = rng.choice(HEADS)
    if op == "lora":
        width = rng.randrange(len(WIDTHS))
        k, ns = WIDTHS[width]
        adapters, rank = _log(rng, 1, 40), rng.choice((8, 16, 24, 32, 64, 128))
        # values of x and y, and products of all adapters with all rows, no more than the listed prompt's
        cap = min(4099 * 32768 // (k + sum(ns)), 4099 * 8 * 64 // (adapters * rank) * 32768 // (k + sum(ns)), 4099)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, max(1, cap)), spread=rng.choice(("packed", "mixed")),
                    requests=_log(rng, 1, 40), adapters=adapters, idle=rng.choice((0, 0, 3, 8)), rank=rank, width=width)
    if op == "rope":
        most = min(16383, 16383 * 40 * 128 // ((hq + heads) * dim))
        return dict(op=op, dtype=dtype, out=rng.choice(("fp32", "fp16", "bf16")), tokens=_log(rng, 1, most), hq=hq, heads=heads, dim=dim,
                    rot=rng.choice((dim, dim, dim // 2)), fused=rng.choice((0, 1)), norm=rng.choice((0, 1)), pairs=rng.choice((0, 1)),
                    base=rng.choice((1e4, 5e5, 1e6)), start=rng.choice((0, _log(rng, 1, 1000000))))
    batch = _log(rng, 1, 64)
    hi = _log(rng, 1, min(12287, int(math.sqrt(12287 ** 2 * 32 * 128 / (batch * hq * dim)))))
    if dtype == "fp32":
        hi = max(1, hi // 2)
    return dict(op=op, dtype=dtype, batch=batch, hq=hq, heads=heads, dim=dim, lo=rng.choice((hi, _log(rng, 1, hi), 0)), hi=hi,
                fused=rng.choice((0, 1)), window=rng.choice((0, 0, 0, _log(rng, 1, hi))))


# ------------------------------------------------------------------ sizes

def _lens(case):
    """Tokens of each sequence: spread over lo..hi, the first the longest."""
    return [case["hi"] - int((case["hi"] - case["lo"] + 0.999) * ((0.6180339887 * b) % 1.0)) for b in range(case["batch"])]


def _pairs(case):
    """(query, key) pairs of one head."""
    w = case["window"]
    return sum(n * (n + 1) // 2 if not w or n <= w else w * (w + 1) // 2 + (n - w) * w for n in _lens(case))


def _ids(case):
    """Each row's adapter: a request's rows behind each other, or rows of all requests in turn; -1 for none."""
    n, r = case["tokens"], min(case["requests"], case["tokens"])
    if case["spread"] == "packed":  # lengths that differ by up to a factor of three
        ends = [sum(2 + (7 * j) % 5 for j in range(i + 1)) for i in range(r)]
        owner = [next(i for i in range(r) if t * ends[-1] < ends[i] * n) for t in range(n)]
    else:
        owner = [(t * 7 + t // 3) % r for t in range(n)]
    ids = [(5 * o + 3) % case["adapters"] for o in owner]
    return [-1 if case["idle"] and t % case["idle"] == case["idle"] - 1 else i for t, i in enumerate(ids)]


def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if case["op"] == "lora":
        k, ns = WIDTHS[case["width"]]
        ids = _ids(case)
        rows, used = sum(i >= 0 for i in ids), len({i for i in ids if i >= 0})
        r, out = case["rank"], sum(ns)
        return {"bytes": max(4, 4 * rows * (k + 2 * out) + used * r * (k * len(ns) + out) * size[case["dtype"]] + 4 * len(ids)),
                "flops": 2 * rows * r * (k * len(ns) + out)}
    if case["op"] == "rope":
        values = case["tokens"] * (case["hq"] + case["heads"]) * case["dim"]
        return {"bytes": values * (size[case["dtype"]] + size[case["out"]]) + 8 * case["tokens"], "flops": 8 * values}
    n = sum(_lens(case))
    return {"bytes": 2 * n * (case["hq"] + case["heads"]) * case["dim"] * size[case["dtype"]] + 4 * case["batch"] + 4,
            "flops": 4 * _pairs(case) * case["hq"] * case["dim"]}


# ----------------------------------------------------------------- inputs

def _rows(tokens, widths, dtype, gen, fused):
    """Rows of normal values, one channel in 32 a few times larger: tensors of their own, or views of one row."""
    x = torch.randn((tokens, sum(widths)), generator=gen, device="cuda")
    x *= 1 + 3 * (torch.rand(x.shape[1], generator=gen, device="cuda") < 1 / 32).float()
    parts = x.to(dtype).split(list(widths), 1)
    return list(parts) if fused else [p.contiguous() for p in parts]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s, dtype = dict(case), DTYPES[case["dtype"]]
    if case["op"] == "lora":
        k, ns = WIDTHS[case["width"]]
        n, r, m = case["adapters"], case["rank"], case["tokens"]
        s["x"] = torch.randn((m, k), generator=gen, device="cuda")
        s["y"] = [torch.randn((m, w), generator=gen, device="cuda") for w in ns]
        s["a"] = [(torch.randn((n, r, k), generator=gen, device="cuda") * k ** -0.5).to(dtype) for _ in ns]
        s["b"] = [(torch.randn((n, w, r), generator=gen, device="cuda") * r ** -0.5).to(dtype) for w in ns]
        s["scales"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
        s["ids"] = torch.tensor(_ids(case), dtype=torch.int32).cuda()
        if own:
            from gguf_quant_integer_gb300 import xq
            s["adapters"] = xq.Adapters([(a, b, s["scales"], 0) for a, b in zip(s["a"], s["b"])])
        return s
    hq, heads, dim = case["hq"], case["heads"], case["dim"]
    widths = (hq * dim, heads * dim, heads * dim)
    if case["op"] == "rope":
        q, k, _ = _rows(case["tokens"], widths, dtype, gen, case["fused"])
        s["q"], s["k"] = q.unflatten(1, (hq, dim)), k.unflatten(1, (heads, dim))
        s["positions"] = case["start"] + torch.arange(case["tokens"], device="cuda")
        if case["norm"]:
            s["qw"], s["kw"] = (1 + 0.3 * torch.randn(dim, generator=gen, device="cuda") for _ in range(2))
        else:
            s["qw"] = s["kw"] = None
        if own:
            from gguf_quant_integer_gb300 import xq
            s["rope"] = xq.Rope(case["rot"], base=case["base"], pairs=bool(case["pairs"]))
        return s
    lens = _lens(case)
    starts = [sum(lens[:b]) for b in range(len(lens) + 1)]
    q, k, v = _rows(starts[-1], widths, dtype, gen, case["fused"])
    s["q"], s["k"], s["v"] = q.unflatten(1, (hq, dim)), k.unflatten(1, (heads, dim)), v.unflatten(1, (heads, dim))
    s["starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
    s["scale"] = 1 / math.sqrt(dim)
    return s


# ------------------------------------------------------------ plain forms

def _plain_lora(s, a, b, y):
    """All adapters' products with all rows, of which a row's own ones are kept."""
    n, r, k = a.shape
    t = (s["x"] @ a.float().flatten(0, 1).T).unflatten(1, (n, r))
    at = torch.arange(n, device=t.device, dtype=torch.int32)
    t = torch.where((s["ids"][:, None] == at)[:, :, None], t * s["scales"][:, None], 0)
    y += t.flatten(1) @ b.float().transpose(1, 2).flatten(0, 1)
    return y


def _plain_rope(s, x, weight):
    rot, dtype = s["rot"], DTYPES[s["out"]]
    x = x.float()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    freq = s["base"] ** (torch.arange(0, rot, 2, device=x.device, dtype=torch.float64) / -rot)
    angle = (s["positions"].double()[:, None] * freq)[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    if s["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1).to(dtype)


def _plain_attn(s):
    """Sequences as a padded batch, all scores at once."""
    hq, heads, dim, most = s["hq"], s["heads"], s["dim"], max(1, s["hi"])
    starts, group, total = s["starts"].long(), hq // heads, s["q"].shape[0]
    lens = starts[1:] - starts[:-1]
    t = torch.arange(most, device=starts.device)
    at = (starts[:-1, None] + t).clamp(max=max(0, total - 1))  # [batch, most]: rows past a sequence's end are masked
    pad = lambda x: x[at].float().transpose(1, 2)  # noqa: E731
    q = (pad(s["q"]) * s["scale"]).unflatten(1, (heads, group)).flatten(2, 3)  # [batch, heads, group * most, dim]
    mask = t <= t[:, None]
    if s["window"]:
        mask = mask & (t > t[:, None] - s["window"])
    scores = (q @ pad(s["k"]).transpose(-1, -2)).unflatten(2, (group, most))
    scores = scores.masked_fill_(~mask, -math.inf)
    p = torch.exp(scores.sub_(scores.amax(-1, keepdim=True)))
    del scores
    out = (p.flatten(2, 3) @ pad(s["v"])).unflatten(2, (group, most)) / p.sum(-1, keepdim=True)
    owner = torch.searchsorted(starts[1:], torch.arange(total, device=starts.device), right=True)
    return out.flatten(1, 2).transpose(1, 2)[owner, torch.arange(total, device=starts.device) - starts[owner]].to(s["q"].dtype)


# -------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if own:
        from gguf_quant_integer_gb300 import xq
        if op == "lora":
            return s["adapters"].add([s["x"]], s["y"], s["ids"])
        if op == "rope":
            q, k = xq.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], s["qw"], s["kw"], eps=EPS, dtype=DTYPES[s["out"]])
            return {"q": q, "k": k}
        return xq.prompt_attn(s["q"], s["k"], s["v"], s["starts"], scale=s["scale"], window=s["window"])
    if op == "lora":
        return [_plain_lora(s, a, b, y) for a, b, y in zip(s["a"], s["b"], s["y"])]
    if op == "rope":
        return {"q": _plain_rope(s, s["q"], s["qw"]), "k": _plain_rope(s, s["k"], s["kw"])}
    return _plain_attn(s)


# ------------------------------------------------- the definition in 64 bits

def _exact_rope(case, x, weight, positions):
    x, half = x.double(), case["rot"] // 2
    if weight is not None:
        x = weight.double() * x * (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).rsqrt()
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       positions.double()[:, None, None] * torch.exp(i.double() * (-2 * math.log(case["base"]) / case["rot"])))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        out = []
        for a, b, y in zip(s["a"], s["b"], s["y"]):
            y = y.double()
            for i in set(_ids(case)) - {-1}:
                rows = torch.nonzero(s["ids"] == i)[:, 0]
                y[rows] += (s["x"][rows].double() @ a[i].double().T) @ b[i].double().T * s["scales"][i].double()
            out.append(y)
        return out
    if case["op"] == "rope":
        return {"q": _exact_rope(case, s["q"], s["qw"], s["positions"]), "k": _exact_rope(case, s["k"], s["kw"], s["positions"])}
    group, window = case["hq"] // case["heads"], case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for n in _lens(case):
        for i in range(0, n, 2048):  # rows i .. e see keys b .. e
            e, b = min(n, i + 2048), max(0, i + 1 - window) if window else 0
            rows, keys = slice(first + i, first + e), slice(first + b, first + e)
            far = torch.arange(i, e, device="cuda")[:, None] - torch.arange(b, e, device="cuda")
            hidden = (far < 0) | (far >= window) if window else far < 0
            for h in range(case["heads"]):
                k, v = s["k"][keys, h].double(), s["v"][keys, h].double()
                q = s["q"][rows, h * group:(h + 1) * group].double().transpose(0, 1)
                z = torch.einsum("gid,jd->gij", q, k).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
                out[rows, h * group:(h + 1) * group] = torch.einsum("gij,jd->gid", torch.softmax(z, -1), v).transpose(0, 1)
        first += n
    return out
