"""mla_plan_chunks at the edges of its arguments' ranges, against the Python
twin (exact)."""

import pytest

from tests.test_gpu_plan import check, mla, random_step  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head,tail", [(1, -2 ** 31), (2 ** 31 - 1, -2 ** 31), (0, -2 ** 31), (-2 ** 31, 2 ** 31 - 1),
                                       (2 ** 31 - 1, 2 ** 31 - 1), (5, -7)])
def test_free_range_whose_difference_wraps(mla, head, tail):  # noqa: F811
    """tail - head leaves 32 bits: the range counts as empty all the same."""
    ctx, new, req, table, free, _, _, num_pages, n = random_step(21, 9, 12, 4, 80, 0)
    check(mla, ctx, new, req, table, free, head, tail, num_pages, n)
