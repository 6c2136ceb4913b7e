"""mla_release_pages on the GPU against the plain form (exact)."""

import random

import numpy as np
import pytest
import torch

from tests import _stay_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


class Case:
    def __init__(self, seed, B, P, move, rows=None, spare=5, front=3):
        r = random.Random(seed)
        cap = P * 64
        self.move, self.rows = move, rows or B + 3
        self.old = [min(cap, r.choice([0, 1, 63, 64, 65, cap, r.randint(0, cap)])) for _ in range(B)]
        self.new = [r.choice([0, o, max(0, o - 1), max(0, o - 64), r.randint(0, o)]) for o in self.old]
        self.req = r.sample(range(self.rows), B)
        used = sum(-(-o // 64) for o in self.old)
        fresh = sum(-(-n // 64) for n, o in zip(self.new, self.old) if n < o) if move else 0
        back = sum(-(-o // 64) - (0 if move else -(-n // 64)) for n, o in zip(self.new, self.old) if n < o)
        ids = list(range(used + fresh + spare))
        r.shuffle(ids)
        self.num_pages = len(ids)
        self.table = np.full((B, P), -1, np.int32)
        for b, o in enumerate(self.old):
            self.table[b, :-(-o // 64)] = [ids.pop() for _ in range(-(-o // 64))]
        self.page_table = np.full((self.rows, P), -7, np.int32)
        self.head = back - fresh + front
        self.free = [-3] * self.head + ids + [-4] * 2
        self.tail = self.head + len(ids)

    def check(self, mla, repeat=1, stream=None):
        pt, free = self.page_table.copy(), list(self.free)
        out, lens, rng, err = R.release(self.old, self.new, self.req, self.table, pt, free, self.head, self.tail, self.num_pages,
                                        self.move)
        e = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
        B, P = self.table.shape
        d_pt, d_free, d_out, d_lens, d_rng, d_err = dev(self.page_table), dev(self.free), e(B, P), e(B), e(2), e(1).zero_()
        ins = dev(self.old), dev(self.new), dev(self.req), dev(self.table), dev([self.head, self.tail])
        torch.cuda.synchronize()
        for _ in range(repeat):
            mla.mla_release_pages(ins[0], ins[1], ins[2] if self.move else None, ins[3], d_pt if self.move else None, d_free, ins[4],
                                  self.num_pages, d_out, d_lens, d_rng, move=self.move, dev_err=d_err, stream=stream)
        torch.cuda.synchronize()
        for x, y in ((d_out, out), (d_lens, lens), (d_rng, rng), (d_free, free), (d_pt, pt)):
            assert np.array_equal(x.cpu().numpy(), np.asarray(y, np.int32))
        assert d_err.item() == err
        return err


@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("B,P", [(1, 1), (1, 700), (2, 3), (33, 17), (300, 9), (1024, 5), (1025, 5), (4096, 33)])
def test_random_requests(mla, B, P, move):
    for seed in (1, 2):
        assert Case(seed * 10000 + B, B, P, move, rows=65536 if B == 4096 else None).check(mla, repeat=1 if move else 2) == 0


@pytest.mark.parametrize("move", [False, True])
def test_exact_fit(mla, move):
    assert Case(3, 40, 8, move, spare=0, front=0).check(mla) == 0


@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("less", [1, 7, 10 ** 6])
def test_too_few_places(mla, move, less):
    c = Case(4, 40, 8, move, front=0)
    cut = min(less, c.head)
    c.free, c.head, c.tail = c.free[cut:], c.head - cut, c.tail - cut
    assert c.check(mla) == 16


@pytest.mark.parametrize("less", [1, 7, 10 ** 6])
def test_too_few_pages(mla, less):
    c = Case(5, 40, 8, True, spare=0)
    c.tail = max(c.head, c.tail - less)
    assert c.check(mla) == 16


@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("head,tail", [(-1, 5), (7, 6), (0, 10 ** 6), (-2 ** 31, 2 ** 31 - 1), (2 ** 31 - 1, -2 ** 31)])
def test_bad_free_range(mla, move, head, tail):
    c = Case(6, 12, 6, move)
    c.head, c.tail = head, tail
    assert c.check(mla) & 2


@pytest.mark.parametrize("move", [False, True])
def test_refused_requests(mla, move):
    c = Case(7, 30, 6, move)
    c.old[1], c.new[3], c.old[5], c.new[7] = -4, -1, 6 * 64 + 1, c.old[7] + 1
    c.old[9], c.new[9] = 2 ** 31 - 1, 2 ** 31 - 1
    c.req[11], c.req[13], c.req[15] = -1, 2 ** 31 - 1, c.req[2]
    assert c.check(mla) & 4


@pytest.mark.parametrize("move", [False, True])
def test_ids_outside_the_pool(mla, move):
    c = Case(8, 30, 6, move)
    c.num_pages //= 2
    assert c.check(mla) & 2


def test_on_another_stream(mla):
    assert Case(9, 30, 6, True).check(mla, stream=torch.cuda.Stream()) == 0


def test_plan_and_release_keep_the_list(mla):
    """Steps of the plan and releases, trimming and moving, in turn: the pages
    in use and the free ones always make up the pool."""
    r = random.Random(10)
    B, P, rows, num_pages = 7, 9, 8, 200
    free, page_table = dev(list(range(num_pages))), torch.full((rows, P), -1, dtype=torch.int32, device="cuda")
    req, rng, ctx = dev(r.sample(range(rows), B)), dev([0, num_pages]), [0] * B
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(40):
        new = [min(r.randint(0, 90), P * 64 - c) for c in ctx]
        n = sum(new)
        table, start, lens, head = e(B, P), e(B + 1), e(B), e(1)
        mla.mla_plan_chunks(dev(ctx), dev(new), req, page_table, free, rng, num_pages, table, start, lens, e(n), e(n), e(n), head,
                            dev_err=err)
        rng = torch.stack([head[0], rng[1]])
        now = [c + m for c, m in zip(ctx, new)]
        cut = [r.randint(max(0, c - 100), c) if r.random() < 0.7 else c for c in now]
        out, got, new_rng = e(B, P), e(B), e(2)
        mla.mla_release_pages(lens, dev(cut), req, table, page_table, free, rng, num_pages, out, got, new_rng, move=step % 2 == 1,
                              dev_err=err)
        torch.cuda.synchronize()
        ctx, rng = got.tolist(), new_rng
        assert err.item() == 0 and ctx == cut
        h, t = rng.tolist()
        pages = out.cpu().numpy()
        used = [int(pages[b, p]) for b in range(B) for p in range(-(-ctx[b] // 64))]
        assert sorted(used + free[h:t].tolist()) == list(range(num_pages))
        rows_now = page_table.cpu().numpy()[req.cpu().numpy()]
        assert all(rows_now[b, p] == pages[b, p] for b in range(B) for p in range(-(-ctx[b] // 64)))
