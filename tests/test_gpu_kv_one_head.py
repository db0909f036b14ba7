"""Rows of a cache of one KV head: the stride between heads has no meaning."""
import pytest
import torch

from test_gpu_kv_cache import xq  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [64, 1, 7, 4096])
def test_any_stride_of_the_only_head(xq, stride):  # noqa: F811
    x = torch.randn(9, 192, device="cuda")
    k, v = (x[:, at:].as_strided((9, 1, 64), (192, stride, 1), at) for at in (64, 128))
    slots = torch.arange(9, device="cuda")
    a, b = xq.KVCache(8, 1, 16, 1, 64), xq.KVCache(8, 1, 16, 1, 64)
    a.write(k, v, slots)
    b.write(k.reshape(9, 1, 64).clone(), v.reshape(9, 1, 64).clone(), slots)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and bool(a.k.any())


def test_strides_that_do_matter_are_checked(xq):  # noqa: F811
    slots = torch.arange(9, device="cuda")
    x = torch.randn(9, 2, 128, device="cuda")
    with pytest.raises(ValueError):
        xq.KVCache(8, 1, 16, 2, 64).write(x[:, :, :64], x[:, :, 64:], slots)
    with pytest.raises(ValueError):
        xq.KVCache(8, 1, 16, 1, 64).write(x[:, :1, ::2], x[:, 1:, ::2], slots)
    with pytest.raises(ValueError):
        xq.KVCache(8, 1, 16, 1, 64).write(x[0, 0], x[0, 0], slots)
