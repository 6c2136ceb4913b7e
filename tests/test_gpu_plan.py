"""mla_plan_chunks on the GPU against the Python twin (exact)."""

import random

import numpy as np
import pytest
import torch

from tests import _step_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def outputs(B, P, n):
    e = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"block_table": e(B, P), "q_start": e(B + 1), "seq_lens": e(B), "positions": e(n), "token_req": e(n),
            "slot": e(n), "free_head": e(1)}


def call(mla, ctx, new, req, table, free, rng, num_pages, out, err, stream=None):
    mla.mla_plan_chunks(ctx, new, req, table, free, rng, num_pages, *[out[k] for k in (
        "block_table", "q_start", "seq_lens", "positions", "token_req", "slot", "free_head")], dev_err=err, stream=stream)


def check(mla, ctx, new, req, table, free, head, tail, num_pages, n, repeat=1):
    B, P = len(ctx), table.shape[1]
    want_table = table.copy()
    want, want_err = R.plan(ctx, new, req, want_table, list(free), head, tail, num_pages, n)
    t, out, err = dev(table), outputs(B, P, n), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(ctx), dev(new), dev(req), t, dev(free), dev([head, tail])
    for _ in range(repeat):
        call(mla, *args, num_pages, out, err)
    torch.cuda.synchronize()
    for k, v in want.items():
        assert np.array_equal(out[k].cpu().numpy(), v), k
    assert np.array_equal(t.cpu().numpy(), want_table)
    assert err.item() == want_err


def random_step(seed, B, rows, P, hi_new, pad, spare=5, zero=0.2):
    r = random.Random(seed)
    cap = P * 64
    new = [0 if r.random() < zero else r.randint(1, min(hi_new, cap)) for _ in range(B)]
    ctx = [r.choice([0, 1, 63, 64, 65, r.randint(0, cap)]) for _ in range(B)]
    ctx = [min(c, cap - m) for c, m in zip(ctx, new)]
    req = r.sample(range(rows), B)
    old = [-(-c // 64) for c in ctx]
    need = sum(-(-(c + m) // 64) for c, m in zip(ctx, new)) - sum(old)
    num_pages = sum(old) + need + spare
    ids = list(range(num_pages))
    r.shuffle(ids)
    table = np.full((rows, P), -5, np.int32)
    for b in range(B):
        table[req[b], :old[b]] = [ids.pop() for _ in range(old[b])]
    free = [-1] * 3 + ids
    return ctx, new, req, table, free, 3, len(free), num_pages, sum(new) + pad


@pytest.mark.parametrize("B,rows,P,hi,pad", [(1, 1, 1, 1, 0), (1, 4, 3, 192, 0), (2, 2, 9, 64, 1), (31, 40, 17, 300, 40),
                                             (33, 64, 16, 5, 0), (513, 600, 33, 40, 7), (4096, 65536, 5, 3, 0),
                                             (4095, 4095, 3, 120, 11)])
def test_random_steps(mla, B, rows, P, hi, pad):
    for seed in (1, 2):
        check(mla, *random_step(100 * B + seed, B, rows, P, hi, pad), repeat=2)


def test_no_tokens_and_empty_requests(mla):
    check(mla, *random_step(5, 7, 9, 4, 3, 0, zero=1.0))
    check(mla, *random_step(6, 7, 9, 4, 3, 5, zero=1.0))


def test_exact_fit_of_the_free_list(mla):
    check(mla, *random_step(8, 40, 50, 6, 200, 0, spare=0))


@pytest.mark.parametrize("short", [1, 2, 9, 10 ** 6])
def test_free_list_too_short(mla, short):
    ctx, new, req, table, free, head, tail, num_pages, n = random_step(9, 40, 50, 6, 200, 0, spare=0)
    check(mla, ctx, new, req, table, free, head, max(head, tail - short), num_pages, n)


@pytest.mark.parametrize("head,tail", [(-1, 5), (7, 6), (0, 1000)])
def test_bad_free_range(mla, head, tail):
    ctx, new, req, table, free, _, _, num_pages, n = random_step(10, 9, 12, 4, 80, 0)
    check(mla, ctx, new, req, table, free, head, tail, num_pages, n)


def test_refused_requests(mla):
    ctx, new, req, table, free, head, tail, num_pages, n = random_step(11, 20, 30, 6, 100, 0)
    ctx, new, req = list(ctx), list(new), list(req)
    ctx[2] = -1
    new[4] = -7
    ctx[6] = 6 * 64 + 1
    new[8], ctx[8] = 2 ** 31 - 1, 2 ** 31 - 1
    req[10] = 30
    req[12] = -3
    req[14] = req[3]
    check(mla, ctx, new, req, table, free, head, tail, num_pages, n)
    check(mla, ctx, new, req, table, free, head, tail, num_pages, n // 2)
    check(mla, ctx, new, req, table, free, head, tail, num_pages, 0)


def test_ids_outside_the_pool(mla):
    ctx, new, req, table, free, head, tail, num_pages, n = random_step(12, 30, 31, 6, 100, 3)
    check(mla, ctx, new, req, table, free, head, tail, num_pages // 2, n)


def test_steps_follow_each_other_in_a_graph(mla):
    """A captured plan replayed with new lengths and the moved head."""
    B, P, rows, n, num_pages = 6, 8, 9, 64, 60
    r = random.Random(3)
    ctx, req = np.zeros(B, np.int64), r.sample(range(rows), B)
    table = np.full((rows, P), -1, np.int32)
    free = list(range(num_pages))
    r.shuffle(free)
    d = dict(ctx=dev(ctx), new=dev(np.zeros(B)), req=dev(req), table=dev(table), free=dev(free), range=dev([0, num_pages]))
    out, err = outputs(B, P, n), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(mla, d["ctx"], d["new"], d["req"], d["table"], d["free"], d["range"], num_pages, out, err)
    head = 0
    for _ in range(9):
        new = [r.randint(0, 10) for _ in range(B)]
        d["ctx"].copy_(dev(ctx))
        d["new"].copy_(dev(new))
        d["range"][0] = head
        g.replay()
        want, want_err = R.plan(list(ctx), new, req, table, free, head, num_pages, num_pages, n)
        torch.cuda.synchronize()
        assert err.item() == want_err == 0
        for k, v in want.items():
            assert np.array_equal(out[k].cpu().numpy(), v), k
        assert np.array_equal(d["table"].cpu().numpy(), table)
        head = int(out["free_head"].item())
        ctx = ctx + np.array(new)


def test_on_another_stream(mla):
    ctx, new, req, table, free, head, tail, num_pages, n = random_step(13, 50, 60, 6, 100, 3)
    want, _ = R.plan(ctx, new, req, table.copy(), free, head, tail, num_pages, n)
    t, out = dev(table), outputs(50, 6, n)
    args = dev(ctx), dev(new), dev(req), t, dev(free), dev([head, tail])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(mla, *args, num_pages, out, None, stream=s)
    s.synchronize()
    assert np.array_equal(out["slot"].cpu().numpy(), want["slot"])
