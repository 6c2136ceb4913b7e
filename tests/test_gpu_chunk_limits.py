"""mla_chunk_attention at the edges of its ranges: many short segments, very
uneven weights, small scales, waits that run out anywhere."""

import time

import pytest
import torch

from tests._helpers import F_INT8
from tests.test_gpu_chunk import Batch, mla  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,B,n", [(128, 40, 65), (64, 60, 129), (16, 300, 66)])
def test_many_short_segments_end_at_once(mla, H, B, n):  # noqa: F811
    """Thousands of one-tile segments: no role is left waiting for a hand-over
    that has passed.  Such a wait would last the limit, 10 seconds; the calls
    take milliseconds."""
    t = Batch(mla, [(0, n)] * B, H, F_INT8, F_INT8)
    ws = t.workspace()
    o = t.call(ws=ws)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(20):
        again = t.call(ws=ws)
        torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 2.0
    assert t.err.item() == 0
    assert torch.equal(o, again)
    t.check(o, seqs=[0, B // 2, B - 1], heads=[0, H - 1])
