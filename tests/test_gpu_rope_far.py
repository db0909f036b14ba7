"""Rotation at far positions, against angles in whole numbers."""
import math

import pytest
import torch

from gguf_quant_integer_gb300 import build as xqbuild
from test_rope_table import BITS, frequencies, two_pi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xq():
    xqbuild.build()
    from gguf_quant_integer_gb300 import xq as _xq
    return _xq


@pytest.mark.parametrize("base,rot", [(1e4, 128), (1e6, 128), (5e5, 64)])
def test_angles_at_far_positions(xq, base, rot):
    """A unit vector's turn is its angle's cosine and sine. The table is off by 2^-65 of a turn a position at most, what the kernel
    keeps by 2^-34 of one (cut off), the two series by 2^-24 of 1 each with their four roundings: 5 of 2^-24."""
    far = [0, 1, 131071, (1 << 20) + 3, (1 << 31) - 1, (1 << 31) + 7, (1 << 36) + 12345, (1 << 40) + 1, -1, -(1 << 33) - 5]
    q = torch.zeros(len(far), 1, 128, device="cuda")
    q[:, :, :rot // 2] = 1.0  # the first elements of all pairs
    got, _ = xq.qk_norm_rope(q, q.clone(), torch.tensor(far, dtype=torch.int64, device="cuda"), xq.Rope(rot, base=base))
    turn = two_pi()
    for i, f in enumerate(frequencies(base, rot)):
        for t, p in enumerate(far):
            angle = float((p * f) % turn) / 2.0 ** BITS
            off = abs(p) * 2.0 ** -65 * 2 * math.pi + 2.0 ** -34 * 2 * math.pi + 5 * 2.0 ** -24
            assert abs(float(got[t, 0, i]) - math.cos(angle)) <= off, (p, i)
            assert abs(float(got[t, 0, i + rot // 2]) - math.sin(angle)) <= off, (p, i)
