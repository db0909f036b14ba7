"""The rotation's table against the definition in whole numbers: base^(-2i / rot) / factor / (2 pi) turns, to 64 bits."""
import math

import pytest

from gguf_quant_integer_gb300 import xq

BITS = 400


def two_pi():
    """2 pi 2^BITS by Euler's series pi / 2 = sum of k! / (3 5 .. (2k + 1))."""
    one = 1 << (BITS + 20)
    term, total, k = one, one, 1
    while term:
        term = term * k // (2 * k + 1)
        total += term
        k += 1
    return total * 4 >> 20


def root(x, n):
    """The whole part of x's n-th root."""
    lo, hi = 0, 1 << (x.bit_length() // n + 1)
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if mid ** n <= x else (lo, mid - 1)
    return lo


def frequencies(base, rot, factors=None):
    """Radians a position, times 2^BITS."""
    num, den = float(base).as_integer_ratio()
    n = rot // 2
    step = root((den << (BITS * n)) // num, n)  # base^(-2 / rot) 2^BITS
    f, out = 1 << BITS, []
    for i in range(n):
        num, den = (float(factors[i]) if factors is not None else 1.0).as_integer_ratio()
        out.append(f * den // num)
        f = f * step >> BITS
    return out


@pytest.mark.parametrize("base,rot,factors", [
    (10000.0, 128, None), (1e6, 128, None), (500000.0, 64, None), (1e4, 96, None), (2.0, 16, None), (0.5, 16, None), (1234567.891, 256, None),
    (1e4, 32, [1 + 0.37 * i for i in range(16)]), (1e6, 16, [1e-20, -2.0, 3.3, 1e6, 8.0, 0.1, 1e-7, 31.0])])
def test_turns_are_right_to_64_bits(base, rot, factors):
    """Rounded to nearest, and the steps of this check's own whole numbers: never more than one unit off."""
    table = xq.Rope(rot, base=base, factors=factors, device="cpu").turns.tolist()
    turn = two_pi()
    assert len(table) == rot // 2
    for got, f in zip(table, frequencies(base, rot, factors)):
        want = ((f << 65) // turn + 1) >> 1
        assert (got - want + 2) % (1 << 64) <= 4 and (got - want + (1 << 63)) % (1 << 64) - (1 << 63) in (-1, 0, 1)


def test_what_has_no_frequencies_is_refused():
    import numpy as np
    for kw in (dict(base=0.0), dict(base=-2.0), dict(base=float("nan")), dict(factors=[0.0] * 8), dict(factors=[float("nan")] * 8), dict(factors=[1.0] * 7)):
        with pytest.raises(ValueError):
            xq.Rope(16, device="cpu", **kw)
    with pytest.raises(ValueError):
        xq.Rope(24, device="cpu")
    assert xq.Rope(0, device="cpu").turns.numel() == 0
    # frequencies that are none: no turn
    assert xq.Rope(16, factors=np.full(8, math.inf), device="cpu").turns.tolist() == [0] * 8
    assert xq.Rope(16, base=math.inf, device="cpu").turns.tolist()[1:] == [0] * 7
    # fp32 factors count as the numbers they are
    f = np.linspace(1, 3, 8, dtype=np.float32)
    assert xq.Rope(16, factors=f, device="cpu").turns.tolist() == xq.Rope(16, factors=f.astype(np.float64), device="cpu").turns.tolist()
