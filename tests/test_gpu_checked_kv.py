"""GPU runs of the checked build's KV cache kernels: the oracle's results, and no check of an access may fail.

Sizes end in every way that the kernels' arithmetic knows: inside and at the end of 16-key steps, tiles and pages, with and
without a join, with windows and prefixes, whole and half row tiles. The sequences' pages are most of a pool, its first and
last among them."""
import pytest

import test_gpu_kv_cache as kv
from test_gpu_checked_build import no_check_failed, xq  # noqa: F401 (the fixture: the checked library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["q8", "q4"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dim,heads,page,tokens,lead", [(128, 8, 64, 1, 0), (64, 3, 16, 33, 0), (96, 1, 128, 200, 3),
                                                        (256, 2, 16, 2000, 1)])
def test_checked_write_and_read(xq, kind, dtype, dim, heads, page, tokens, lead):  # noqa: F811
    kv.test_write_stores_the_defined_bytes_and_read_returns_their_values(xq, kind, dtype, dim, heads, page, tokens, lead)


@pytest.mark.parametrize("kind,dtype", kv.KINDS)
@pytest.mark.parametrize("heads,group,dim,page,n_q,lens,window,prefix", [
    (2, 4, 128, 16, 1, [1, 0, 15, 16, 17, 63, 64, 65, 130, 257], 0, 0),
    (1, 8, 256, 32, 3, [3, 1, 700, 0, 37], 0, 0),
    (2, 5, 96, 16, 1, [300, 6001], 0, 0),
    (3, 1, 64, 64, 70, [70, 49, 333, 2000], 50, 0),
    (2, 4, 64, 32, 1, [1, 0, 17, 5], 0, 100),
    (2, 7, 128, 32, 9, [9, 20, 3, 0, 64], 0, 1513),
    (1, 6, 96, 16, 1, list(range(1, 40)), 0, 257),
    (1, 2, 256, 16, 2, [2, 90], 0, 2000)])
def test_checked_attention(xq, kind, dtype, heads, group, dim, page, n_q, lens, window, prefix):  # noqa: F811
    kv.attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, window=window, prefix=prefix, seed=n_q + dim)


@pytest.mark.parametrize("kind,dtype", [("q8", "bf16"), ("q8", "fp16"), ("q4", "bf16"), ("q4", "fp16")])
@pytest.mark.parametrize("heads,group,dim,page,n_q,lens,window,prefix", [
    (2, 4, 128, 64, 1, [1 + i % 9 for i in range(128)], 0, 3001),        # two row tiles, whole
    (8, 4, 128, 16, 1, [1 + i % 9 for i in range(25)], 0, 4001),         # most of one
    (1, 13, 96, 16, 3, [5, 0, 40, 3, 2, 1] * 3, 0, 6000),                # chunks of which the last is not full
    (2, 4, 128, 64, 300, [1400, 299, 1, 0, 777], 0, 0),
    (2, 2, 96, 32, 400, [1003, 2050], 700, 0),
    (4, 1, 64, 128, 127, [2900, 2000, 126], 0, 0)])
def test_checked_attention_on_row_tiles(xq, kind, dtype, heads, group, dim, page, n_q, lens, window, prefix):  # noqa: F811
    kv.attention_case(xq, kind, dtype, heads, group, dim, page, n_q, lens, window=window, prefix=prefix, seed=n_q + dim)


def test_checked_bad_indices(xq):  # noqa: F811
    kv.test_bad_slots_are_skipped_and_recorded(xq)
    kv.test_bad_pages_and_lengths_are_masked_and_recorded(xq)
    kv.test_row_tiles_with_bad_pages_and_odd_scales(xq, "fp16")
    no_check_failed(xq)


def test_checked_workspaces(xq):  # noqa: F811
    """Workspaces of exactly the size asked for, other calls' records in them."""
    kv.test_other_stream_and_own_workspace(xq)
    kv.test_repeated_calls_agree_bit_for_bit(xq)
    no_check_failed(xq)
