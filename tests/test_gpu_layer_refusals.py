"""A layer call with adapters that is refused has written nothing."""
import pytest
import torch

from gguf_quant_integer_gb300 import synth
from test_gpu_lora import adapters, some_ids, xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


def test_refused_before_the_projections_run(xq):  # noqa: F811
    projs = (synth.Proj("q", synth.Q4_K, 512, 256, 0), synth.Proj("down", synth.Q6_K, 768, 512, 1))
    ws = [synth.gen_weight(p.qtype, 40 + t, p.N, p.K) for t, p in enumerate(projs)]
    good = {0: adapters(3, 16, 512, 256, "bf16"), 1: adapters(3, 8, 768, 512, "fp16")}
    M = 20
    inputs = [torch.randn(M, 512, device="cuda"), torch.randn(M, 768, device="cuda")]
    ids = some_ids(M, 3)
    odd = torch.zeros(3 * 16 * 512 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 16, 512)  # not on a 16-byte boundary
    layer = xq.Layer(projs, ws, M, adapters=good)
    misplaced = xq.Layer(projs, ws, M, adapters={0: (odd, *good[0][1:])})
    for y in (*layer.y, *misplaced.y):
        y.fill_(7.0)
    bad = ((ids.long(), inputs), (ids[:M - 1], inputs), (ids.cpu(), inputs), (torch.stack([ids, ids], 1)[:, 0], inputs),
           (ids, [inputs[0].half(), inputs[1]]), (ids, inputs[:1]), (ids, [inputs[0], inputs[1][:, :512]]))
    for i, x in bad:
        with pytest.raises((ValueError, xq.XQError)):
            layer.forward(x, ids=i)
    with pytest.raises(xq.XQError):
        misplaced.forward(inputs, ids=ids)
    torch.cuda.synchronize()
    assert all(bool((y == 7.0).all()) for y in (*layer.y, *misplaced.y))
    layer.forward(inputs, ids=ids)
    assert all(not bool((y == 7.0).all()) for y in layer.y)
