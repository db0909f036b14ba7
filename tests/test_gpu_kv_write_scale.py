"""The Q8_0 scale's rounding: fp16 of the fp32 quotient max|x| / 127, not of a product with 1 / 127 rounded to fp32.

The two differ by one fp16 step for four significands of the block's largest element, in every binade."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_oracle as ko
from test_gpu_kv_cache import xq  # noqa: F401 (the fixture)

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIGNIFICANDS = (0x7E1FC1, 0x7E9EC1, 0x7F1DC1, 0x7F9CC1)


def blocks():
    """Rows of two blocks [n, 1, 64] whose largest elements have these significands, of both signs, in several binades."""
    rng = np.random.default_rng(0)
    rows = []
    for binade in (-9, -3, -1, 0, 1, 4, 17):  # fp16 scales from a subnormal one up
        for m in SIGNIFICANDS:
            top = np.array((127 + binade) << 23 | m, np.uint32).view(np.float32)
            for sign in (1, -1):
                x = rng.uniform(-1, 1, (1, 64)).astype(np.float32) * top
                x[0, [3, 60]] = sign * top, -sign * top
                rows.append(x)
    return np.stack(rows)


def plain_form():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_cases_tell_the_two_roundings_apart():
    top = np.abs(blocks()).reshape(-1, 32).max(-1)
    product = (top * (np.float32(1) / np.float32(127))).astype(np.float16)
    normal = top / 127 >= 2.0 ** -14
    assert normal.any() and np.all((product != (top / np.float32(127)).astype(np.float16))[normal])


@gpu
def test_plain_form_kernel_and_oracle_store_the_same_blocks(xq):  # noqa: F811
    x = blocks()
    codes, d = ko.quantize(x, ko.Q8_0)
    t = torch.from_numpy(x).cuda()
    plain_codes, plain_d = plain_form()._quantize(t, 8)
    assert np.array_equal(plain_d.cpu().numpy().view(np.uint16), d.view(np.uint16))
    assert np.array_equal(plain_codes.cpu().numpy(), codes)
    n = len(x)
    cache, pool = xq.KVCache(ko.Q8_0, -(-n // 16), 16, 1, 64), ko.Pool(ko.Q8_0, -(-n // 16), 16, 1, 64)
    cache.write(t, t, torch.arange(n, device="cuda"))
    for s in range(n):
        pool.put(s, x[s])
    assert np.array_equal(cache.k.cpu().numpy(), pool.raw) and np.array_equal(cache.v.cpu().numpy(), pool.raw)
