"""GPU runs of the checked build's adapters, norms with rotation and prompt attention: 64-bit results, and no check may fail.

Sizes end in every way that the kernels' arithmetic knows: inside and at the end of row tiles, key tiles and 32-column blocks,
rows of no sequence and of no adapter, one row and whole jobs of 16, 32 and 64."""
import pytest

import test_gpu_lora as lora
import test_gpu_prompt_attn as attn
import test_gpu_qk_rope as rope
from test_gpu_checked_build import no_check_failed, xq  # noqa: F401 (the fixture: the checked library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,n,rank,K,N", [(1, 3, 16, 4096, 4096), (7, 4, 64, 512, 130), (33, 5, 128, 256, 1000), (64, 64, 8, 1024, 515),
                                          (700, 7, 40, 1536, 77), (1000, 4, 64, 512, 2048)])
def test_checked_adapters(xq, dtype, M, n, rank, K, N):  # noqa: F811
    lora.run(xq, M, [lora.adapters(n, rank, K, N, dtype)], lora.some_ids(M, n))
    no_check_failed(xq)


def test_checked_bad_adapters(xq):  # noqa: F811
    lora.test_ids_that_no_adapter_has(xq)
    no_check_failed(xq)


@pytest.mark.parametrize("dtype,out", [("fp32", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("T,H,Hk,D,rot,pairs", [(1, 32, 8, 128, 128, False), (257, 5, 1, 64, 64, True), (33, 3, 1, 96, 48, False),
                                                (7, 1, 1, 256, 64, True)])
def test_checked_norm_and_rotation(xq, dtype, out, T, H, Hk, D, rot, pairs):  # noqa: F811
    rope.case(xq, T, H, Hk, D, rot, pairs, dtype, out, fused=True, lead=3)
    no_check_failed(xq)


@pytest.mark.parametrize("dtype", attn.KINDS)
@pytest.mark.parametrize("H,Hk,D,window", [(4, 1, 128, 0), (7, 1, 64, 100), (2, 2, 96, 0), (6, 3, 256, 0), (5, 1, 256, 130)])
def test_checked_prompt_attention(xq, dtype, H, Hk, D, window):  # noqa: F811
    attn.case(xq, [1, 0, 2, 31, 33, 0, 64, 127, 128, 129, 255, 300, 600], H, Hk, D, dtype, window=window, first=3, behind=5)
    no_check_failed(xq)


def test_checked_bad_sequences(xq):  # noqa: F811
    attn.test_bad_bounds_are_left_out_and_recorded(xq)
    no_check_failed(xq)
