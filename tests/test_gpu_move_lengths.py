"""mla_move_tokens: lengths that are equal but no lengths are reported, as any that do not fit."""

import numpy as np
import pytest
import torch

from tests._helpers import F_INT8
from tests.test_gpu_select_move import dev, fill, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


@pytest.mark.parametrize("length,bad", [(-1, True), (-2 ** 31, True), (8 * 64 + 1, True), (2 ** 31 - 1, True), (0, False), (1, False),
                                        (200, False), (8 * 64, False)])
def test_equal_lengths(mla, length, bad):
    """A sequence of all its tokens stays where it is, also with more of them than max_keep; the others' tokens move."""
    lens, new = [100, length, 90], [50, length, 40]
    src, n1 = tables([100, 512, 90], 8, 1)
    dst, num_pages = tables([50, 512, 40], 8, 2, first=n1)
    kept = np.tile(np.arange(0, 100, 2, dtype=np.int32), (3, 1))
    kept[2, :40] = np.arange(40)
    cache = fill(mla, F_INT8, F_INT8, num_pages, 3)
    before = cache.pool.cpu().numpy().reshape(num_pages, -1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_move_tokens(cache, dev(src), dev(lens), dev(kept), dev(new), dev(dst), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == (4 if bad else 0)
    after = cache.pool.cpu().numpy().reshape(num_pages, -1)
    changed = set(np.nonzero((before != after).any(1))[0].tolist())
    assert changed == {int(dst[0, 0]), int(dst[2, 0])}
