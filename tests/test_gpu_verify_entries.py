"""mla_verify_drafts where a row's entries are not probabilities: infinite
entries of one of the two rows alone, and finite ones whose sum no fp32 holds
(exact: whole numbers)."""

import pytest
import torch

from tests.test_gpu_verify import INF, NAN, TYPES, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


class Pair(Step):
    """A step whose draft rows lie `apart` elements further apart than the target's."""

    def __init__(self, *args, apart=0, **kw):
        super().__init__(*args, **kw)
        self.apart = apart

    def placed(self, t):
        if t is None:
            return None
        wide = torch.full((t.shape[0], self.vocab + (self.apart if t is self.draft else 0)), NAN, dtype=t.dtype, device="cuda")
        wide[:, : self.vocab] = t.cuda()
        return wide[:, : self.vocab]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("apart", [0, 1, 8])
@pytest.mark.parametrize("vocab", [4, 5000, 5003])
def test_an_infinite_entry_of_the_draft_row_alone(mla, dtype, apart, vocab):
    """c(q) is 0 there, so the token keeps all of the target's weight."""
    for at in (0, 1, vocab // 2, vocab - 1):
        s = Pair([3, 2, 2, 1], vocab, dtype, seed=vocab + at, apart=apart)
        s.target *= 0.5
        s.target[:, at] = 0.5
        s.draft[:, at] = INF
        s.u_acc[:] = NAN                                   # the first draft is rejected
        for u in (0.02, 0.3, 0.6, 0.99):
            s.u_samp[:] = u
            s.check(mla)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("apart", [0, 1])
def test_an_infinite_entry_holds_all_that_is_left(mla, dtype, apart):
    s = Pair([2, 2], 3000, dtype, seed=1, apart=apart)
    s.draft = s.target.clone()
    s.draft[0, 1700], s.draft[2, 2999] = INF, INF
    s.u_acc[:] = NAN
    assert s.check(mla)[1][:, 0].tolist() == [1700, 2999]


@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("lookup", [False, True])
def test_sums_that_no_fp32_holds(mla, dtype, apart, lookup):
    """Rows need not add up to 1: here entries up to 3e38, thousands of them, alone and against a draft's."""
    for seed in range(3):
        s = Pair([3, 2, 1, 1], 4100, dtype, lookup=lookup, seed=seed, apart=apart)
        g = torch.Generator().manual_seed(seed)
        s.target = (3e38 * torch.rand(s.target.shape, generator=g)).to(dtype)
        if not lookup:
            s.draft = (2e38 * torch.rand(s.target.shape, generator=g)).to(dtype)
        s.u_acc[:] = 1.0
        s.check(mla)


def test_one_sum_in_a_lane_too_large(mla):
    """Two entries of one lane's, each finite, their sum not; an infinite and a NaN beside them."""
    s = Pair([1, 1, 1], 2048, seed=7)
    s.draft = None
    s.target[:, 8] = s.target[:, 10] = 3e38
    s.target[1, 9], s.target[1, 11] = INF, NAN
    s.u_samp = torch.tensor([0.2, 0.7, 1.0])
    assert s.check(mla)[1][:2, 0].tolist() == [8, 10]
