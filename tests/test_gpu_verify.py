"""mla_verify_drafts on the GPU against the plain form (exact: whole numbers)."""

import random

import numpy as np
import pytest
import torch

from tests import _stay_reference as R

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def ints(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


class Step:
    def __init__(self, counts, vocab, dtype=torch.float32, lookup=False, seed=0, width=None, stride=None, close=0.5):
        g = torch.Generator().manual_seed(seed)
        self.counts, self.B, self.n, self.vocab = counts, len(counts), sum(counts), vocab
        self.start = [sum(counts[:b]) for b in range(self.B + 1)]
        self.width = max(1, max(counts)) if width is None else width
        logits = 2 * torch.randn((self.n, vocab), generator=g)
        self.target = torch.softmax(logits, -1).to(dtype)
        q = torch.softmax(logits + close * torch.randn((self.n, vocab), generator=g), -1)
        self.draft = None if lookup else q.to(dtype)
        self.drafts = torch.multinomial(q, 1, generator=g)[:, 0].int() if self.n else torch.zeros(0, dtype=torch.int32)
        self.u_acc = torch.rand(self.n, generator=g)
        self.u_samp = torch.rand(self.B, generator=g)
        self.lens = [50 + c for c in counts]
        self.stride = stride

    def placed(self, t):
        """t on the GPU, with the row stride asked for (what lies between rows is NaN)."""
        if t is None or self.stride is None:
            return None if t is None else t.cuda()
        wide = torch.full((t.shape[0], self.stride), NAN, dtype=t.dtype, device="cuda")
        wide[:, : self.vocab] = t.cuda()
        return wide[:, : self.vocab]

    def args(self, mla, err):
        e = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
        out = e(self.B), e(self.B, self.width), e(self.B)
        return (self.placed(self.target), self.placed(self.draft), self.drafts.cuda(), ints(self.start), self.u_acc.cuda(),
                self.u_samp.cuda(), out[0], out[1]), dict(seq_lens=ints(self.lens), kept_lens=out[2], dev_err=err), out

    def check(self, mla, stream=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        a, kw, out = self.args(mla, err)
        torch.cuda.synchronize()
        mla.mla_verify_drafts(*a, **kw, stream=stream)
        torch.cuda.synchronize()
        draft = None if self.draft is None else self.draft.double().numpy()
        want = R.verify(self.target.double().numpy(), draft, self.drafts.numpy(), self.start, self.u_acc.numpy(),
                        self.u_samp.numpy(), self.width, self.lens)
        for name, x, y in zip(("accepted", "tokens", "kept_lens"), out, want):
            assert np.array_equal(x.cpu().numpy(), y), name
        assert err.item() == want[3]
        return want


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 7, 1023, 1024, 1025, 32003, 131072])
def test_vocabularies_types(mla, dtype, lookup, vocab):
    Step([5, 1, 3, 0, 2], vocab, dtype, lookup, seed=vocab).check(mla)


@pytest.mark.parametrize("counts", [[1], [2], [9], [0], [300], [3] * 150, [1, 0, 0, 8] * 20], ids=lambda c: "%dx%d" % (len(c), max(c)))
def test_batches(mla, counts):
    for seed in (1, 2):
        Step(counts, 501, seed=seed).check(mla)


def test_largest_batch(mla):
    r = random.Random(5)
    Step([r.randint(0, 3) for _ in range(4096)], 61, seed=3).check(mla)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("stride", [2000, 2003, 2048])
def test_row_strides(mla, dtype, stride):
    Step([4, 4, 2], 2000, dtype, seed=4, stride=stride).check(mla)


def test_views_off_a_vector_boundary(mla):
    """The rows begin 4 bytes behind a 16-byte boundary, the draft's 8."""
    s = Step([3, 2], 4099, seed=5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, kw, out = s.args(mla, err)
    t, q = torch.empty(5 * 4099 + 1, device="cuda"), torch.empty(5 * 4099 + 2, device="cuda")
    t[1:], q[2:] = a[0].flatten(), a[1].flatten()
    mla.mla_verify_drafts(t[1:].view(5, 4099), q[2:].view(5, 4099), *a[2:], **kw)
    want = R.verify(s.target.double().numpy(), s.draft.double().numpy(), s.drafts.numpy(), s.start, s.u_acc.numpy(),
                    s.u_samp.numpy(), s.width, s.lens)
    assert np.array_equal(out[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("lookup", [False, True])
def test_all_pass_and_none_pass(mla, lookup):
    s = Step([6, 6], 700, lookup=lookup, seed=6)
    s.u_acc[:] = 0.0
    assert list(s.check(mla)[0]) == [5, 5]
    s.u_acc[:] = NAN
    assert list(s.check(mla)[0]) == [0, 0]


def test_borders_of_exact_sums(mla):
    """Probabilities in sixteenths: u = k / 16 lies exactly on a border, and belongs to the token behind it."""
    p = torch.zeros(17, 40)
    for i in range(16):
        p[:, 2 * i + 3] = 1 / 16
    s = Step([1] * 17, 40, seed=7)
    s.target, s.u_samp = p, torch.tensor([k / 16 for k in range(17)])
    s.draft = None
    want = s.check(mla)
    assert [int(x) for x in want[1][:, 0]] == [2 * min(k, 15) + 3 for k in range(17)]


def test_u_outside_the_interval(mla):
    s = Step([1] * 6, 300, seed=8)
    s.u_samp = torch.tensor([0.0, 1.0, 1.5, -2.0, NAN, INF])
    s.check(mla)


def test_accept_at_the_border_is_exact(mla):
    """u q == p rejects, one step less accepts."""
    s = Step([2, 2, 2], 8, seed=9)
    s.drafts[:] = 3
    s.target[:, 3], s.draft[:, 3] = 0.25, 0.5
    s.u_acc = torch.tensor([0.5, 0, np.nextafter(np.float32(0.5), np.float32(0)), 0, np.nextafter(np.float32(0.5), np.float32(1)), 0])
    assert list(s.check(mla)[0]) == [0, 1, 0]


def test_equal_rows_leave_nothing_to_resample(mla):
    s = Step([2, 2], 500, seed=10)
    s.draft = s.target.clone()
    s.u_acc[:] = 1.0                                       # u q == p: rejected with w = 0 everywhere
    assert list(s.check(mla)[0]) == [0, 0]


def test_not_probabilities(mla):
    """NaN, infinite and negative entries have no weight; rows need not add up to 1."""
    s = Step([3, 2, 1], 2100, seed=11)
    s.target *= 7.5
    s.draft[:, 5:40] = NAN
    s.target[:, 100:120] = NAN
    s.target[:, 300], s.draft[:, 301] = INF, INF
    s.target[:, 400:500] *= -1
    s.check(mla)


def test_rows_without_weight(mla):
    s = Step([2, 1, 1], 900, seed=12)
    s.target[:3] = 0.0
    s.target[1] = NAN
    assert s.check(mla)[3] == 32


def test_drafts_outside_the_vocabulary(mla):
    for lookup in (False, True):
        s = Step([3, 3, 3], 100, lookup=lookup, seed=13)
        s.u_acc[:] = 0.0
        s.drafts[0], s.drafts[4], s.drafts[8] = -1, 100, 2 ** 31 - 1        # the last is not used
        assert s.check(mla)[3] == 32


def test_refused_sequences(mla):
    assert Step([3, 5, 2], 100, seed=14, width=4).check(mla)[3] == 4
    for start in ([0, 5, 3, 10], [-1, 3, 8, 10], [0, 3, 8, 11]):
        s = Step([3, 5, 2], 100, seed=15)
        s.start = start
        assert s.check(mla)[3] == 4
    s = Step([3, 5, 2], 100, seed=16)
    s.lens = [1, 0, -5]
    s.u_acc[:] = NAN
    assert s.check(mla)[3] == 4


def test_lengths_in_place_and_none(mla):
    s = Step([3, 5, 2], 1000, seed=17)
    a, kw, out = s.args(mla, None)
    mla.mla_verify_drafts(*a)
    lens = ints(s.lens)
    want = s.check(mla)
    mla.mla_verify_drafts(*a, seq_lens=lens, kept_lens=lens)
    assert np.array_equal(lens.cpu().numpy(), want[2]) and np.array_equal(out[1].cpu().numpy(), want[1])


def test_on_another_stream_and_in_a_graph(mla):
    s = Step([3, 5, 2], 5000, seed=18)
    s.check(mla, stream=torch.cuda.Stream())
    a, kw, out = s.args(mla, None)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        mla.mla_verify_drafts(*a, **kw)
    for seed in range(3):
        t = Step([3, 5, 2], 5000, seed=20 + seed)
        for x, y in zip(a[:2] + a[2:3] + a[4:6], (t.target, t.draft, t.drafts, t.u_acc, t.u_samp)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        want = R.verify(t.target.double().numpy(), t.draft.double().numpy(), t.drafts.numpy(), t.start, t.u_acc.numpy(),
                        t.u_samp.numpy(), t.width, t.lens)
        for x, y in zip(out, want):
            assert np.array_equal(x.cpu().numpy(), y)


def test_the_drawn_tokens_follow_the_target(mla):
    """Accepted and redrawn first tokens together are distributed as the
    target's row, whatever the draft model: 20000 independent sequences, each
    token's count within 6 standard deviations of its expectation."""
    g = torch.Generator().manual_seed(19)
    p, q = torch.softmax(torch.randn(12, generator=g), -1), torch.softmax(torch.randn(12, generator=g), -1)
    total = 20000
    counts = torch.zeros(12, dtype=torch.long)
    for part in range(5):
        B = total // 5
        e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        drafts = torch.zeros(2 * B, dtype=torch.int32)
        drafts[0::2] = torch.multinomial(q, B, replacement=True, generator=g).int()
        acc, tok = e(B), e(B, 2)
        mla.mla_verify_drafts(p.expand(2 * B, 12).contiguous().cuda(), q.expand(2 * B, 12).contiguous().cuda(), drafts.cuda(),
                              torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda"), torch.rand(2 * B, generator=g).cuda(),
                              torch.rand(B, generator=g).cuda(), acc, tok)
        counts += torch.bincount(tok[:, 0].long().cpu(), minlength=12)
    sd = (total * p * (1 - p)).sqrt()
    assert ((counts - total * p).abs() <= 6 * sd).all()
