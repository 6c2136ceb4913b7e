"""mla_plan_chunks at the edges of its arguments' ranges, against the Python
twin (exact)."""

import os
import subprocess
import sys

import pytest

from tests.test_gpu_plan import check, mla, random_step  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("head,tail", [(1, -2 ** 31), (2 ** 31 - 1, -2 ** 31), (0, -2 ** 31), (-2 ** 31, 2 ** 31 - 1),
                                       (2 ** 31 - 1, 2 ** 31 - 1), (5, -7)])
def test_free_range_whose_difference_wraps(mla, head, tail):  # noqa: F811
    """tail - head leaves 32 bits: the range counts as empty all the same."""
    ctx, new, req, table, free, _, _, num_pages, n = random_step(21, 9, 12, 4, 80, 0)
    check(mla, ctx, new, req, table, free, head, tail, num_pages, n)


@pytest.mark.parametrize("batch,rows", [(2341, 2341), (2345, 2345), (2354, 2354), (2330, 4096), (1580, 65536)])
def test_shared_memory_near_the_default_limit(batch, rows):
    """Batches whose tables just fit 48 KB of shared memory beside nothing
    else: served by a process that has made no larger call before."""
    run = ("from tests.test_gpu_plan import check, random_step; import mla_latent_kv_append_gb300 as mla; "
           "check(mla, *random_step(3, %d, %d, 3, 2, 1))" % (batch, rows))
    r = subprocess.run([sys.executable, "-c", run], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
