"""Adapters, norms with rotation and prompt attention in 64 bits, with how far off a kernel may be.

Bounds count roundings: a value of type t is rounded by at most finfo(t).eps / 2 of itself (U), fp32 sums of n products by
n times that of the sum of their magnitudes. Nothing here uses the package."""
import math

import torch

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a subnormal step


def attention(q, k, v, starts, scale, window=0):
    """(o, bound) of packed prompts; rows of no sequence are None-like (NaN). q [T, H, D], k and v [T, Hk, D]."""
    dtype, (T, H, D), Hk = q.dtype, q.shape, k.shape[1]
    g = H // Hk
    o = torch.full((T, H, D), math.nan, dtype=torch.float64, device=q.device)
    bound = o.clone()
    for b in range(len(starts) - 1):
        s, e = starts[b], starts[b + 1]
        n = e - s
        if n <= 0:
            continue
        qd, kd, vd = (x[s:e].double() for x in (q, k, v))
        i = torch.arange(n, device=q.device)
        far = i[:, None] - i
        hidden = (far < 0) | (far >= window) if window else far < 0
        for h in range(H):
            kk, vv = kd[:, h // g], vd[:, h // g]
            z = (qd[:, h] @ kk.T * scale).masked_fill(hidden, -math.inf)
            top = z.amax(-1, keepdim=True)
            w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            w = w / w.sum(-1, keepdim=True)
            seen = torch.where(hidden[:, :, None], 0.0, vv[None]) if n <= 64 else None  # 0 * NaN of unseen keys stays out
            o[s:e, h] = (w[:, :, None] * seen).sum(1) if seen is not None else w @ vv
            # a score is off by the rounding of D products and sums (a tensor core cuts off instead: a whole step), of the
            # scale and of the exponent's argument and function (4 ulp of its size and 4 of the result)
            dz = ((qd[:, h].abs() @ kk.abs().T * abs(scale)) * (2 * D + 8) * 2.0 ** -24 + 8 * 2.0 ** -24).masked_fill(hidden, 0.0)
            dz = torch.nan_to_num(dz).amax(-1, keepdim=True)
            mag = w @ torch.nan_to_num(vv.abs())
            # numerator and denominator both move by dz; weights are rounded to the type of V; sums of n terms
            rel = 2 * dz + (U[dtype] if dtype != torch.float32 else 2.0 ** -21) + (2 * n + 8) * 2.0 ** -24
            bound[s:e, h] = mag * rel * (1 + U[dtype]) + o[s:e, h].abs() * U[dtype] + TINY[dtype] + mag.amax() * n * 2.0 ** -30
    return o, bound


def norm_rope(x, positions, base, rot, pairs, weight, eps, out, magnitude=1.0, factors=None):
    """(y, bound) of heads' rows x [T, H, D]."""
    xd, D = x.double(), x.shape[-1]
    r = xd if weight is None else xd * weight.double() / torch.sqrt(xd.square().mean(-1, keepdim=True) + eps)
    i = torch.arange(rot // 2, device=x.device)
    freq = base ** (-2.0 * i.double() / max(rot, 1))
    if factors is not None:
        freq = freq / torch.as_tensor(factors, dtype=torch.float64, device=x.device)
    turn = torch.remainder(positions.double()[:, None] * freq, 2 * math.pi)[:, None]
    a, b = (r[..., 0:rot:2], r[..., 1:rot:2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:rot])
    ya, yb = a * turn.cos() - b * turn.sin(), b * turn.cos() + a * turn.sin()
    y, size = r.clone(), r.abs()
    size2 = a.abs() + b.abs()
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya * magnitude, yb * magnitude
        size[..., 0:rot:2] = size[..., 1:rot:2] = size2 * abs(magnitude)
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ya * magnitude, yb * magnitude
        size[..., :rot // 2] = size[..., rot // 2:rot] = size2 * abs(magnitude)
    # the norm: the sum of D squares (D / 2 relative, of the root), mean, root, reciprocal, two products; the turn: the
    # angle's 2^-33 half turns and its rounding, 2 ulp of sine and cosine, the magnitude, two products, a sum; this
    # oracle's own angle, position * freq in 64 bits
    far = float(positions.abs().max()) * 2.0 ** -52 if positions.numel() else 0.0
    rel = ((D / 2 + 6 if weight is not None else 0) + 10) * 2.0 ** -24 + far
    return y, size * rel + (y.abs() + size * rel) * U[out] + TINY[out]


def lora(x, a, b, scales, ids, y):
    """(y + what the adapters add, bound) for fp32 rows x [M, K]."""
    want, bound = y.double(), torch.zeros_like(y, dtype=torch.float64)
    K, R = x.shape[1], a.shape[1]
    for i in sorted(set(ids.tolist())):
        if not 0 <= i < a.shape[0]:
            continue
        rows = torch.nonzero(ids == i)[:, 0]
        s = 1.0 if scales is None else float(scales[i].double())
        A, B, X = a[i].double(), b[i].double(), x[rows].double()
        t = X @ A.T
        want[rows] += s * (t @ B.T)
        # both products: operands as two tf32 numbers each (2^-22 each, one of them is dropped), sums of fp32 whose terms may
        # be cut off instead of rounded; the scale; the sum with y
        dt = (X.abs() @ A.abs().T) * (2.0 ** -20 + (K + 8) * 2.0 ** -23)
        mag = t.abs() @ B.abs().T
        bound[rows] = abs(s) * (dt @ B.abs().T + mag * (2.0 ** -20 + (R + 8) * 2.0 ** -23)) + want[rows].abs() * 2.0 ** -24
    return want, bound


def within(got, want, bound, what=""):
    got = got.double()
    live = ~torch.isnan(want)
    off = (got - want).abs() - bound
    bad = live & ~((off <= 0) | (got == want))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {want.numel()} off, by up to {float(torch.nan_to_num(off[bad], nan=math.inf).max()):.3g}; first at {torch.nonzero(bad)[0].tolist()}"


def rms(got, want):
    live = ~torch.isnan(want)
    g, w = got.double()[live], want[live]
    return float(((g - w).square().sum() / w.square().sum().clamp(min=1e-300)).sqrt())
