"""xq_device_error for callers that use no KV cache costs what its own kernels' records cost."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own: which records are read depends on what the process has launched. Times are the least of several
# rounds, in units of a 4-byte copy from the device, so that they do not depend on the machine. The matmul kernels' records
# are two copies each way; the KV cache's, read for everyone, were some twenty more.
SCRIPT = """
import sys, time
sys.path.insert(0, sys.argv[1])
from gguf_quant_integer_gb300 import build, xq
build.build()
import torch
word = torch.zeros(1, dtype=torch.int32, device="cuda")
host = torch.zeros(1, dtype=torch.int32)

def least(f):
    best = 1e9
    for _ in range(20):
        t = time.perf_counter()
        for _ in range(20):
            f()
        best = min(best, (time.perf_counter() - t) / 20)
    return best

copy = least(lambda: host.copy_(word))
alone = least(xq.device_error)
cache = xq.KVCache(8, 1, 16, 1, 64)
cache.read(torch.tensor([99], device="cuda"))  # past the cache: recorded
assert xq.device_error() == (3 << 8) | 1 and xq.device_error() == 0
print(copy * 1e6, alone * 1e6, alone / copy)
"""


def test_without_a_kv_cache(tmp_path):
    f = tmp_path / "cost.py"
    f.write_text(SCRIPT)
    r = subprocess.run([sys.executable, str(f), ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    print(r.stdout)
    assert float(r.stdout.split()[-1]) <= 8, r.stdout
