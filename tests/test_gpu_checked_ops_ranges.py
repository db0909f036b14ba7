"""GPU runs of the checked build: adapters with more jobs than clusters, infinities, and prompt attention over several runs of key
tiles and with bounds out of order. 64-bit results, and no check may fail."""
import pytest

import test_gpu_lora_many_jobs as jobs
import test_gpu_lora_non_finite as odd
import test_gpu_prompt_bounds as bounds
import test_gpu_prompt_precision as runs
from test_gpu_checked_build import no_check_failed, xq  # noqa: F401 (the fixture: the checked library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [jobs.SIZES[1], jobs.SIZES[4], jobs.SIZES[5], jobs.SIZES[7]])
@pytest.mark.parametrize("spread", ["own", "uneven"])
def test_checked_more_jobs_than_clusters(xq, dtype, size, spread):  # noqa: F811
    jobs.test_more_jobs_than_clusters(xq, dtype, *size, spread)
    no_check_failed(xq)


@pytest.mark.parametrize("where", ["x", "a", "b"])
def test_checked_infinities(xq, where):  # noqa: F811
    odd.test_infinities(xq, "fp32", 700, 24, 96, 130, where)
    no_check_failed(xq)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_checked_bounds_out_of_order(xq, dtype):  # noqa: F811
    for starts, T in bounds.BOUNDS:
        bounds.test_bounds_out_of_order(xq, dtype, 128, starts, T, 0)
    no_check_failed(xq)


@pytest.mark.parametrize("D", [128, 256])
def test_checked_runs_of_tiles(xq, D):  # noqa: F811
    runs.test_sums_over_runs_of_tiles(xq, "bf16", D, 0.0)
    no_check_failed(xq)
