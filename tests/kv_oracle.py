"""The quantized KV cache and its attention in numpy, from the definitions: blocks, pages and sums in 64 bits.

Shares nothing with the library. Block arithmetic that decides a stored code
(the scale's rounding to fp16, the fp32 quotient) is done in those types, as
the definition fixes them; everything after it is float64.
"""
import numpy as np

Q8_0, Q4_0 = 8, 2
BITS = {Q8_0: 8, Q4_0: 4}


def quantize(x, qtype):
    """x [..., dim] -> codes [..., dim * bits / 8] as stored, scales fp16 [..., dim / 32]."""
    x = np.asarray(x, np.float32)
    x = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(all="ignore"):
        if qtype == Q8_0:
            d = (np.max(np.abs(x), -1) / np.float32(127)).astype(np.float16)
        else:
            first = np.argmax(np.abs(x), -1)
            d = (np.take_along_axis(x, first[..., None], -1)[..., 0] / np.float32(-8)).astype(np.float16)
        w = d.astype(np.float32)[..., None]
        y = np.where(w != 0, x / np.where(w != 0, w, 1), 0).astype(np.float32)
    y = np.where(np.isnan(y), 0, y).astype(np.float64)
    q = np.sign(y) * np.floor(np.abs(y) + 0.5)
    if qtype == Q8_0:
        q = np.clip(q, -127, 127).astype(np.int64) + 128
        return q.astype(np.uint8).reshape(q.shape[:-2] + (-1,)), d
    q = (np.clip(q, -8, 7) + 8).astype(np.uint8)
    b = q[..., :16] | (q[..., 16:] << 4)
    return b.reshape(b.shape[:-2] + (-1,)), d


def values(codes, scales, qtype):
    """float64 values of stored blocks."""
    if qtype == Q8_0:
        c = codes.reshape(codes.shape[:-1] + (-1, 32)).astype(np.float64) - 128
    else:
        b = codes.reshape(codes.shape[:-1] + (-1, 16))
        c = np.concatenate((b & 15, b >> 4), -1).astype(np.float64) - 8
    with np.errstate(invalid="ignore"):
        v = c * scales.astype(np.float64)[..., None]
    return v.reshape(v.shape[:-2] + (-1,))


class Pool:
    """One pool's bytes, with row access by (slot, head)."""

    def __init__(self, qtype, n_pages, page_size, heads, dim, fill=0):
        self.qtype, self.page, self.heads, self.dim = qtype, page_size, heads, dim
        self.row = dim * BITS[qtype] // 8
        self.size = heads * page_size * (self.row + dim // 16)
        self.raw = np.full(n_pages * self.size, fill, np.uint8)

    def _at(self, slot, h):
        line = h * self.page + slot % self.page
        base = slot // self.page * self.size
        return base + line * self.row, base + self.heads * self.page * self.row + line * (self.dim // 16)

    def put(self, slot, x):
        """x [heads, dim]"""
        codes, d = quantize(x, self.qtype)
        for h in range(self.heads):
            c, s = self._at(slot, h)
            self.raw[c:c + self.row] = codes[h]
            self.raw[s:s + self.dim // 16] = d[h].view(np.uint8)

    def rows(self, slots):
        """float64 [len(slots), heads, dim]"""
        n, r, s2 = len(slots), self.row, self.dim // 16
        if n == 0:
            return np.zeros((0, self.heads, self.dim))
        slots = np.asarray(slots, np.int64)
        line = np.arange(self.heads)[None] * self.page + (slots % self.page)[:, None]
        base = (slots // self.page * self.size)[:, None]
        c = (base + line * r)[..., None] + np.arange(r)
        s = (base + self.heads * self.page * r + line * s2)[..., None] + np.arange(s2)
        return values(self.raw[c], np.ascontiguousarray(self.raw[s]).view(np.float16), self.qtype)


def attention(q, k, v, scale, n_q_pos, window=0):
    """q [n_q, hq, dim], k and v [n, heads, dim] float64, n_q_pos: position of each query token.
    Returns out, and for error bounds sum_j p_j |v_j| and the largest scale * sum_d |q_d k_jd| of the visible keys,
    both broadcast to out's shape, and the number of visible keys."""
    n_q, hq, dim = q.shape
    heads = k.shape[1]
    g = hq // heads
    out, absum, smax = np.zeros((3, n_q, hq, dim))
    keys = np.zeros((n_q, 1, 1), np.int64)
    q = np.asarray(q, np.float64)
    for i in range(n_q):
        end = min(n_q_pos[i] + 1, k.shape[0])
        start = max(0, n_q_pos[i] + 1 - window) if window else 0
        if end <= start:
            continue
        keys[i] = end - start
        for h in range(hq):
            kk, vv = k[start:end, h // g], v[start:end, h // g]
            z = kk @ q[i, h] * scale
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h] = p @ vv
            absum[i, h] = p @ np.abs(vv)
            smax[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, absum, smax, keys


def tolerance(out, absum, smax, keys, dtype):
    """Largest error of an attention output that its arithmetic allows (dtype: "fp32", "fp16", "bf16").

    A relative error e of the products q_d k_jd moves a score by at most e * S, S = scale * sum_d |q_d k_jd|, and every
    softmax weight by a factor within exp(+-2 e S); a relative error f of the weighted terms p_j v_jd moves the output by
    at most f * sum_j p_j |v_jd|.
      fp32: q and the weights as two fp16 numbers each (error 2^-22), block sums of at most 8 blocks and a few products
        in fp32 (a tensor-core sum may cut off instead of rounding: 2^-23 a step): e = 2^-22 + 24 * 2^-23. The sum over
        keys advances in steps of 16 keys, each within 2^-23 of it, and merges of parts: f = 2^-22 + (keys / 16 + 40) * 2^-23.
        exp2 of scores and their differences: 4 ulp, plus the score's own rounding, 2^-23 * S.
      16-bit: keys and values may enter as fp16 numbers (2^-11), weights as one fp16 number: e = 2^-10, f = 2^-10 + the
        fp32 terms; the result is rounded once (2^-11 or 2^-8, or half the least fp16 step).
    """
    steps = (keys / 16 + 40) * 2.0 ** -23
    e, f = (2.0 ** -22 + 25 * 2.0 ** -23, 2.0 ** -22) if dtype == "fp32" else (2.0 ** -10, 2.0 ** -10)
    t = absum * (np.expm1(2 * e * smax) + f + steps + 4 * 2.0 ** -23)
    if dtype == "fp32":
        return t + 2.0 ** -24 * np.abs(out) + 1e-30
    return t + (2.0 ** -11 if dtype == "fp16" else 2.0 ** -8) * (np.abs(out) + t) + 2.0 ** -25
