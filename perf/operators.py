"""Timed cases of the quantized KV cache: writing it, reading it back, and the attention that reads it.

Three operators over one paged cache (K and V as Q8_0 or Q4_0 blocks of 32 values):

  write   quantize new K and V rows into their slots, then read the same rows back as floats
  read    read the rows of a set of slots back as floats
  attn    attention of the last n_q tokens of each sequence over its own pages (causal, grouped heads)
  shared  the same for a batch whose sequences all begin with one prefix, which is stored once

A pool (one for K, one for V) is n_pages pages of bytes. A page holds the codes of its tokens,
[heads][page_size][dim * bits / 8] bytes, then their scales, fp16 [heads][page_size][dim / 32].
A value is d * (code - 128) with 8-bit codes and d * (code - 8) with 4-bit ones; byte j of a 4-bit
block holds element j in its low half and element j + 16 in its high half.
Token slot s is row s % page_size of page s // page_size.

`own` selects what run() calls: this package's kernels, or the same mathematics as elementary
torch operations in fp32.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BITS = {"q8": 8, "q4": 4}
# Query heads, KV heads and head size of an attention layer: the 8B-class layer (4096 and 1024 wide q and k/v
# projections), the 1.5B-class one (1536 and 256 wide), and generic ones with other groupings and head sizes.
HEADS = ((32, 8, 128), (12, 2, 128), (8, 8, 64), (14, 2, 64), (16, 16, 96), (24, 3, 128), (16, 2, 256), (5, 1, 64))


def listed():
    return [
        # One new token of one sequence, as every decode step writes it: a call of almost no work.
        dict(name="write_token_q8_fp32", op="write", type="q8", dtype="fp32", tokens=1, heads=8, dim=128, page=64, fused=0),
        # The step of a wide decode batch with a 4-bit cache, K and V taken as views of one qkv row.
        dict(name="write_batch_q4_bf16", op="write", type="q4", dtype="bf16", tokens=257, heads=2, dim=128, page=32, fused=12),
        # A long prompt written in one call, in the fp32 that the projections give.
        dict(name="write_prompt_q8_fp32", op="write", type="q8", dtype="fp32", tokens=16383, heads=8, dim=128, page=64, fused=0),
        # A short prefix taken out of the cache, to be worked on in floats.
        dict(name="read_prefix_q8_fp32", op="read", type="q8", dtype="fp32", tokens=1001, heads=8, dim=128, page=64),
        # A whole long conversation read back from a 4-bit cache.
        dict(name="read_long_q4_bf16", op="read", type="q4", dtype="bf16", tokens=65536, heads=8, dim=128, page=64),
        # The first steps of a single chat: latency is all.
        dict(name="attn_short_q8_fp32", op="attn", type="q8", dtype="fp32", batch=1, n_q=1, hq=32, heads=8, dim=128, page=64,
             lo=97, hi=97, idle=0, window=0),
        # An ordinary decode batch, sequences of all lengths, one batch entry in seven idle.
        dict(name="attn_batch_q8_fp32", op="attn", type="q8", dtype="fp32", batch=64, n_q=1, hq=32, heads=8, dim=128, page=64,
             lo=211, hi=8192, idle=7, window=0),
        # One user with a very long context on a 4-bit cache.
        dict(name="attn_long_q4_bf16", op="attn", type="q4", dtype="bf16", batch=1, n_q=1, hq=32, heads=8, dim=128, page=64,
             lo=131071, hi=131071, idle=0, window=0),
        # Five tokens a sequence: four drafted ones and the last accepted one, 1.5B-class heads.
        dict(name="attn_drafts_q8_fp16", op="attn", type="q8", dtype="fp16", batch=16, n_q=5, hq=12, heads=2, dim=128, page=32,
             lo=300, hi=4099, idle=0, window=0),
        # A few users of one system prompt.
        dict(name="shared_small_q8_fp32", op="shared", type="q8", dtype="fp32", batch=8, n_q=1, hq=32, heads=8, dim=128, page=64,
             prefix=1000, lo=5, hi=61),
        # Many answers from one long document, bf16 queries.
        dict(name="shared_large_q8_bf16", op="shared", type="q8", dtype="bf16", batch=64, n_q=1, hq=32, heads=8, dim=128, page=64,
             prefix=32768, lo=1, hi=512),
        # The same in fp32 on a 4-bit cache with six query heads a KV head; the prefix ends inside a page.
        dict(name="shared_odd_q4_fp32", op="shared", type="q4", dtype="fp32", batch=48, n_q=1, hq=12, heads=2, dim=128, page=32,
             prefix=6001, lo=1, hi=333),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn", "shared"))
    hq, heads, dim = rng.choice(HEADS)
    case = dict(op=op, type=rng.choice(("q8", "q4")), dtype=rng.choice(("fp32", "fp16", "bf16")), heads=heads, dim=dim,
                page=rng.choice((16, 32, 64, 128)))
    width = heads * dim
    if op == "write":
        case.update(tokens=_log(rng, 1, min(16383, 16383 * 1024 // width)), fused=rng.choice((0, hq)))
    elif op == "read":
        case.update(tokens=_log(rng, 1, min(65536, 65536 * 1024 // width)))
    else:
        most = 64 * 4096 * 1024 // width  # values of K that a batch may hold: the listed batch's
        batch = _log(rng, 1, 64)
        n_q = rng.choice((1, 1, 1, 2, 3, 5, 8, _log(rng, 9, 128)))
        cap = min(131071, most // batch, (1 << 32) // (dim * batch * n_q * hq))  # also bounds the products' size
        hi = max(n_q, _log(rng, 1, max(cap, 1)))
        if op == "attn":
            lo = rng.choice((hi, min(hi, _log(rng, n_q, max(hi, n_q)))))
            case.update(batch=batch, n_q=n_q, hq=hq, lo=lo, hi=hi, idle=rng.choice((0, 0, 5)),
                        window=rng.choice((0, 0, 0, _log(rng, 1, max(hi, 1)))))
        else:
            hi = min(hi, 700 + n_q)
            case.update(batch=batch, n_q=n_q, hq=hq, prefix=_log(rng, 1, min(32768, max(1, cap))), lo=min(hi, n_q), hi=hi)
    return case


# ------------------------------------------------------------------ sizes

def _lens(case):
    """Tokens of each sequence's own pages (the query tokens among them): spread over lo..hi, the first the longest."""
    lens = [case["hi"] - int((case["hi"] - case["lo"] + 0.999) * ((0.6180339887 * b) % 1.0)) for b in range(case["batch"])]
    every = case.get("idle", 0)
    return [0 if every and b % every == every - 1 else n for b, n in enumerate(lens)]


def _row_bytes(case):
    """Code and scale bytes of one token's K (or V) row of one head."""
    return case["dim"] * BITS[case["type"]] // 8 + case["dim"] // 16


def _seen(case):
    """(key, query) pairs of one head, and the keys that any query of their sequence sees, in own pages and in the prefix."""
    n_q, window, prefix = case["n_q"], case.get("window", 0), case.get("prefix", 0)
    pairs = keys = 0
    for n in _lens(case):
        first = n
        for i in range(n_q):
            end = n + prefix - n_q + i + 1
            start = max(0, end - window) if window else 0
            pairs += max(0, end - start)
            first = min(first, start)
        keys += max(0, n - first) if not prefix else n
    return pairs, keys


def work(case):
    size = {"fp32": 4, "fp16": 2, "bf16": 2}[case["dtype"]]
    row = _row_bytes(case)
    if case["op"] in ("write", "read"):
        rows = 2 * case["tokens"] * case["heads"]  # of K and V
        if case["op"] == "read":
            return {"bytes": rows * (row + case["dim"] * size) + 8 * case["tokens"], "flops": 2 * rows * case["dim"]}
        # the input read, the blocks written, then read again and given back in fp32
        return {"bytes": rows * (case["dim"] * size + 2 * row + 4 * case["dim"]) + 16 * case["tokens"],
                "flops": 6 * rows * case["dim"]}
    pairs, keys = _seen(case)
    keys += case.get("prefix", 0)
    out = case["batch"] * case["n_q"] * case["hq"] * case["dim"]
    return {"bytes": 2 * keys * case["heads"] * row + 2 * out * size + 4 * (keys // case["page"] + case["batch"]),
            "flops": 4 * pairs * case["hq"] * case["dim"]}


# ----------------------------------------------------------------- inputs

def _sizes(case, n_pages):
    return n_pages, case["heads"], case["page"], case["dim"], BITS[case["type"]]


def _views(pool, sizes):
    """Codes [pages][heads][page_size][bytes] and scales [pages][heads][page_size][dim / 32] of a pool, as views."""
    n_pages, heads, page, dim, bits = sizes
    rows = pool.view(n_pages, -1)
    split = heads * page * dim * bits // 8
    return (rows[:, :split].unflatten(1, (heads, page, dim * bits // 8)),
            rows[:, split:].view(torch.float16).unflatten(1, (heads, page, dim // 32)))


def _pool(sizes, gen, spread):
    """A pool full of blocks as real K or V rows give them: normal codes, scales that differ by channel block and token."""
    n_pages, heads, page, dim, bits = sizes
    pool = torch.empty(n_pages * heads * page * (dim * bits // 8 + dim // 16), dtype=torch.uint8, device="cuda")
    codes, scales = _views(pool, sizes)
    top = 127 if bits == 8 else 7
    at = 0
    step = max(1, (1 << 25) // (heads * page * dim))  # pages made at once
    while at < n_pages:
        n = min(step, n_pages - at)
        c = torch.randn((n, heads, page, dim), generator=gen, device="cuda").mul_(top / 2.4).round_().clamp_(-top - (bits == 4), top)
        c = c.add_(128 if bits == 8 else 8).to(torch.uint8)
        if bits == 4:
            c = c.unflatten(3, (dim // 32, 2, 16))
            c = (c[..., 0, :] | (c[..., 1, :] << 4)).flatten(3)
        codes[at:at + n] = c
        block = 0.5 + torch.rand((1, heads, 1, dim // 32), generator=gen, device="cuda")
        token = 0.7 + 0.6 * torch.rand((n, heads, page, 1), generator=gen, device="cuda")
        scales[at:at + n] = (block * token * (spread * 2.4 / top)).half()
        at += n
    return pool


def _activations(tokens, heads, dim, dtype, gen):
    """K or V rows: normal, with one channel in 32 a few times larger, as projections of trained layers have them."""
    x = torch.randn((tokens, heads * dim), generator=gen, device="cuda")
    x *= 1 + 4 * (torch.rand(heads * dim, generator=gen, device="cuda") < 1 / 32).float()
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    heads, dim, page = case["heads"], case["dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        sizes = _sizes(case, -(-n // page) + 2)
        s["sizes"] = sizes
        s["kpool"], s["vpool"] = _pool(sizes, gen, 1.0), _pool(sizes, gen, 1.0)
        order = torch.randperm(sizes[0], generator=gen, device="cuda")[:-(-n // page)]
        slots = (order[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
        s["slots"] = slots[:n].contiguous()
        if case["op"] == "write":
            if case["fused"]:  # one row of query heads, then K, then V
                width = heads * dim
                qkv = _activations(n, case["fused"] + 2 * heads, dim, dtype, gen)
                s["k"] = qkv[:, -2 * width:-width].unflatten(1, (heads, dim))
                s["v"] = qkv[:, -width:].unflatten(1, (heads, dim))
            else:
                s["k"] = _activations(n, heads, dim, dtype, gen).view(n, heads, dim)
                s["v"] = _activations(n, heads, dim, dtype, gen).view(n, heads, dim)
    else:
        lens, prefix = _lens(case), case.get("prefix", 0)
        pages = [-(-n // page) for n in lens]
        head = -(-prefix // page)
        sizes = _sizes(case, sum(pages) + head + 1)
        s["sizes"] = sizes
        s["kpool"], s["vpool"] = _pool(sizes, gen, 1.0), _pool(sizes, gen, 1.0)
        order = torch.randperm(sizes[0], generator=gen, device="cuda").cpu().numpy().astype(np.int32)
        table = np.full((len(lens), max(1, max(pages))), -1, np.int32)  # entries past a sequence's length are not read
        at = head
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        s["pages"] = torch.from_numpy(table).cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if prefix:
            s["prefix_pages"] = torch.from_numpy(order[:head].copy()).cuda()
        s["scale"] = 1 / math.sqrt(dim)
        s["q"] = torch.randn((case["batch"], case["n_q"], case["hq"], dim), generator=gen, device="cuda").to(dtype)
    if own:
        from gguf_quant_integer_gb300 import xq
        n_pages, heads, page, dim, bits = sizes
        s["cache"] = xq.KVCache(xq.XQ_TYPE_Q8_0 if bits == 8 else xq.XQ_TYPE_Q4_0, n_pages, page, heads, dim, k=s["kpool"], v=s["vpool"])
    return s


# ------------------------------------------------------------ plain forms

def _half_away(x):
    """x rounded to whole numbers, halves away from zero."""
    a = x.abs()
    whole = a.floor()
    return torch.copysign(whole + (a - whole >= 0.5).float(), x)


def _quantize(x, bits):
    """Blocks of 32 along the last axis: codes as stored bytes, and fp16 scales."""
    x = x.float().unflatten(-1, (-1, 32))
    size = x.abs()
    if bits == 8:
        # by a number on the device: a CUDA tensor divided by a Python number is multiplied by its rounded reciprocal, which
        # takes four fp32 significands to the neighbouring fp16 scale
        d = (size.amax(-1) / torch.full((), 127.0, device=x.device)).half()
    else:
        d = (x.gather(-1, size.argmax(-1, keepdim=True)).squeeze(-1) / -8).half()
    wide = d.float()[..., None]
    q = _half_away(torch.where(wide != 0, x / wide, 0))
    if bits == 8:
        return (q.clamp(-127, 127) + 128).to(torch.uint8).flatten(-2), d
    q = (q.clamp(-8, 7) + 8).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d


def _values(codes, scales, bits):
    """fp32 values of stored codes [..., bytes] and scales [..., blocks]."""
    if bits == 8:
        c = codes.float().unflatten(-1, (-1, 32)) - 128
    else:
        c = codes.unflatten(-1, (-1, 16))
        c = torch.cat((c & 15, c >> 4), -1).float() - 8
    return (c * scales.float()[..., None]).flatten(-2)


def _plain_write(s):
    page, bits = s["page"], s["sizes"][4]
    at, row = s["slots"] // page, s["slots"] % page
    for pool, x in ((s["kpool"], s["k"]), (s["vpool"], s["v"])):
        codes, scales = _views(pool, s["sizes"])
        c, d = _quantize(x, bits)
        codes[at, :, row] = c
        scales[at, :, row] = d
    return _plain_read(s, torch.float32)


def _plain_read(s, dtype):
    page, bits = s["page"], s["sizes"][4]
    at, row = s["slots"] // page, s["slots"] % page
    (kc, kd), (vc, vd) = _views(s["kpool"], s["sizes"]), _views(s["vpool"], s["sizes"])
    return {"k": _values(kc[at, :, row], kd[at, :, row], bits).to(dtype), "v": _values(vc[at, :, row], vd[at, :, row], bits).to(dtype)}


def _gather(pool, sizes, pages):
    """fp32 rows [..., heads, tokens, dim] of a page table [..., pages]."""
    codes, scales = _views(pool, sizes)
    pages = pages.long()
    x = _values(codes[pages], scales[pages], sizes[4])  # [..., pages, heads, page, dim]
    return x.transpose(-4, -3).flatten(-3, -2)


def _weights(scores, mask):
    """exp(score - the row's largest) where the mask allows, and 0 elsewhere and in rows it leaves empty."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True)
    return torch.exp(scores - torch.where(top == -math.inf, 0, top))


def _plain_attn(s):
    hq, heads, n_q, dim = s["hq"], s["heads"], s["n_q"], s["dim"]
    batch, group = s["q"].shape[0], hq // heads
    # query rows by KV head: [batch, heads, n_q * group, dim]
    q = s["q"].float().view(batch, n_q, heads, group, dim).transpose(1, 2).reshape(batch, heads, n_q * group, dim) * s["scale"]
    keys, vals = _gather(s["kpool"], s["sizes"], s["pages"]), _gather(s["vpool"], s["sizes"], s["pages"])
    prefix = s.get("prefix", 0)
    lens = s["lens"].long()
    # each row's position, counted from the first token of its own pages
    pos = (lens[:, None] - n_q + torch.arange(n_q, device=lens.device)).repeat_interleave(group, 1)[:, None, :, None]
    j = torch.arange(keys.shape[2], device=lens.device)
    mask = (j <= pos) & (j < lens[:, None, None, None])
    if s.get("window", 0):
        mask = mask & (j > pos - s["window"])
    scores = q @ keys.transpose(-1, -2)
    if not prefix:
        p = _weights(scores, mask)
        out = p @ vals
        total = p.sum(-1, keepdim=True)
    else:
        pk, pv = _gather(s["kpool"], s["sizes"], s["prefix_pages"]), _gather(s["vpool"], s["sizes"], s["prefix_pages"])
        i = torch.arange(pk.shape[1], device=lens.device)
        before = (i < prefix) & (i <= pos + prefix)
        flat = q.transpose(0, 1).flatten(1, 2)  # [heads, batch * rows, dim]: one product for the whole batch
        first = (flat @ pk.transpose(-1, -2)).unflatten(1, (batch, n_q * group)).transpose(0, 1)
        p = _weights(torch.cat((first, scores), -1), torch.cat((before.expand_as(first), mask.expand_as(scores)), -1))
        own_part = p[..., pk.shape[1]:] @ vals
        shared_part = p[..., :pk.shape[1]].transpose(0, 1).flatten(1, 2) @ pv
        out = own_part + shared_part.unflatten(1, (batch, n_q * group)).transpose(0, 1)
        total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, out / total, 0)
    return out.view(batch, heads, n_q, group, dim).transpose(1, 2).reshape(batch, n_q, hq, dim).to(s["q"].dtype)


# -------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if not own:
        return _plain_write(s) if op == "write" else _plain_read(s, DTYPES[s["dtype"]]) if op == "read" else _plain_attn(s)
    cache = s["cache"]
    if op == "write":
        cache.write(s["k"], s["v"], s["slots"])
        k, v = cache.read(s["slots"], torch.float32)
        return {"k": k, "v": v}
    if op == "read":
        k, v = cache.read(s["slots"], DTYPES[s["dtype"]])
        return {"k": k, "v": v}
    if op == "attn":
        return cache.attn(s["q"], s["pages"], s["lens"], scale=s["scale"], window=s["window"])
    return cache.attn_shared(s["q"], s["prefix_pages"], s["prefix"], s["pages"], s["lens"], scale=s["scale"])


# ------------------------------------------------- the definition in 64 bits

def _rows64(pool, case, slots):
    """Rows [tokens, heads, dim] of token slots in 64 bits, each byte fetched by its offset in the pool."""
    heads, page, dim, bits = case["heads"], case["page"], case["dim"], BITS[case["type"]]
    row, blocks = dim * bits // 8, dim // 32
    size = heads * page * (row + 2 * blocks)
    line = (slots % page)[:, None] + page * torch.arange(heads, device=slots.device)  # row of the page: [tokens, heads]
    base = (slots // page * size)[:, None, None]
    e = torch.arange(dim, device=slots.device)
    if bits == 8:
        code = pool[base + line[..., None] * row + e].double() - 128
    else:
        byte = pool[base + line[..., None] * row + e // 32 * 16 + e % 16].long()
        code = torch.where(e % 32 < 16, byte % 16, byte // 16).double() - 8
    where = base + heads * page * row + (line[..., None] * blocks + e // 32) * 2
    bits16 = pool[where].long() + 256 * pool[where + 1].long()
    return code * bits16.to(torch.int16).view(torch.float16).double()


def _blocks64(x, bits):
    """The values that rows x [..., dim] stand for after quantization, in 64 bits (the scale rounded to its fp16)."""
    x = x.double().unflatten(-1, (-1, 32))
    if bits == 8:
        d, top, low = x.abs().amax(-1, keepdim=True) / 127, 127, -127
    else:
        big, least = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
        at = torch.arange(32, device=x.device)
        first = torch.where(x.abs() == torch.maximum(big, -least), at, 32).amin(-1, keepdim=True)
        d, top, low = x.gather(-1, first) / -8, 7, -8
    d = d.half().double()
    q = torch.where(d != 0, x / d, 0.0)
    q = torch.sign(q) * torch.floor(q.abs() + 0.5)
    return (q.clamp(low, top) * d).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        bits = BITS[case["type"]]
        return {"k": _blocks64(s["k"], bits), "v": _blocks64(s["v"], bits)}
    if case["op"] == "read":
        return {"k": _rows64(s["kpool"], case, s["slots"]), "v": _rows64(s["vpool"], case, s["slots"])}
    page, n_q, heads, dim = case["page"], case["n_q"], case["heads"], case["dim"]
    group, prefix, window = case["hq"] // heads, case.get("prefix", 0), case.get("window", 0)
    table = s["pages"].long()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = torch.arange(0, dtype=torch.int64, device="cuda")
    if prefix:
        t = torch.arange(prefix, device="cuda")
        at = s["prefix_pages"].long()[t // page] * page + t % page
    kp, vp = _rows64(s["kpool"], case, at), _rows64(s["vpool"], case, at)
    for b, n in enumerate(_lens(case)):
        t = torch.arange(n, device="cuda")
        slots = table[b][t // page] * page + t % page
        k = torch.cat((kp, _rows64(s["kpool"], case, slots)))
        v = torch.cat((vp, _rows64(s["vpool"], case, slots)))
        for i in range(n_q):
            end = prefix + n - n_q + i + 1
            start = max(0, end - window) if window else 0
            if end <= start:
                continue
            q = s["q"][b, i].double().view(heads, group, dim)
            z = torch.einsum("hgd,lhd->hgl", q, k[start:end]) * s["scale"]
            z = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            out[b, i] = torch.einsum("hgl,lhd->hgd", z, v[start:end]).reshape(case["hq"], dim)
    return out
