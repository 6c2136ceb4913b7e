"""mla_select_tokens and mla_move_tokens on the GPU against the plain forms
(exact: positions, and stored bits)."""

import random

import numpy as np
import pytest
import torch

from tests import _stay_reference as R
from tests._helpers import ALL_FORMATS, F_BF16, F_I8OUT, F_INT4, F_INT8, F_INT4S, FMT_NAME, read_tokens

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
EVERY = ALL_FORMATS + [(F_I8OUT, F_BF16), (F_I8OUT, F_INT8)]


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def tables(lens, P, seed, spare=2, first=0):
    r = random.Random(seed)
    pages = [-(-t // 64) for t in lens]
    ids = list(range(first, first + sum(pages) + spare))
    r.shuffle(ids)
    t = np.full((len(lens), P), -1, np.int32)
    for b, n in enumerate(pages):
        t[b, :n] = [ids.pop() for _ in range(n)]
    return t, first + sum(pages) + spare


def check_select(mla, mass, num_pages, table, lens, keep, sinks, recent, max_keep, stream=None):
    want = R.select(mass, num_pages, table, lens, keep, sinks, recent, max_keep)
    B = len(lens)
    kept, out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, max_keep), (B,))]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = torch.from_numpy(mass).cuda(), dev(table), dev(lens), dev(keep)
    torch.cuda.synchronize()
    mla.mla_select_tokens(*args, kept, out, sinks=sinks, recent=recent, dev_err=err, stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want[1])
    assert np.array_equal(kept.cpu().numpy(), want[0])
    assert err.item() == want[2]
    return want[2]


def weights(n, seed, kind):
    g = np.random.RandomState(seed)
    if kind == "spread":
        return (g.rand(n).astype(np.float32) ** -0.7 - 1).astype(np.float32)
    if kind == "zeros":
        m = g.rand(n).astype(np.float32)
        return np.where(m < 0.8, np.float32(0), m)
    if kind == "few":
        return g.choice(np.array([0, -0.0, 1e-40, 1.5, 2.5], np.float32), n)
    m = g.randn(n).astype(np.float32) * 10
    m[g.randint(0, n, n // 7)] = NAN
    m[g.randint(0, n, n // 9)] = INF
    m[g.randint(0, n, n // 9)] = -INF
    m[g.randint(0, n, n // 5)] = -0.0
    return m


@pytest.mark.parametrize("kind", ["spread", "zeros", "few", "odd"])
@pytest.mark.parametrize("lens", [[1], [2], [63, 64, 65], [1000], [40, 999, 5000, 0, 1], [20000]], ids=str)
def test_select(mla, kind, lens):
    P = max(1, -(-max(lens) // 64)) + 1
    table, num_pages = tables(lens, P, 1)
    mass = weights(num_pages * 64, 2, kind)
    r = random.Random(3)
    for sinks, recent in ((0, 0), (4, 33), (1000, 1000)):
        keep = [r.choice([0, 1, t, t + 5, max(0, t - 1), t // 2, t // 16]) for t in lens]
        check_select(mla, mass, num_pages, table, lens, keep, sinks, recent, max(1, max(keep)))


@pytest.mark.parametrize("L", [32768, 32769, 100000, 300000, 500000])
def test_select_over_several_blocks(mla, L):
    """Up to 8 blocks share a sequence, and behind 8 x 49152 tokens weights are read again."""
    lens = [L, 100, L // 2 + 7]
    table, num_pages = tables(lens, -(-L // 64), 4)
    for kind in ("spread", "zeros"):
        mass = weights(num_pages * 64, 5, kind)
        check_select(mla, mass, num_pages, table, lens, [L // 4, 50, L // 3], 4, 64, L // 2)


def test_select_largest_batch(mla):
    r = random.Random(6)
    lens = [r.randint(0, 200) for _ in range(4096)]
    table, num_pages = tables(lens, 4, 7)
    check_select(mla, weights(num_pages * 64, 8, "few"), num_pages, table, lens, [r.randint(0, 200) for _ in lens], 2, 5, 200)


def test_select_sinks_then_recent(mla):
    lens = [500] * 6
    table, num_pages = tables(lens, 9, 9)
    mass = weights(num_pages * 64, 10, "spread")
    check_select(mla, mass, num_pages, table, lens, [3, 4, 5, 10, 13, 14], 4, 9, 20)
    check_select(mla, mass, num_pages, table, lens, [3, 4, 5, 10, 13, 14], 2 ** 31 - 1, 2 ** 31 - 1, 20)


def test_select_refusals(mla):
    lens, keep = [300, 300, -1, 6 * 64 + 1, 300, 300], [-1, 41, 5, 5, 20, 2 ** 31 - 1]
    table, num_pages = tables([300] * 6, 6, 11)
    mass = weights(num_pages * 64, 12, "spread")
    assert check_select(mla, mass, num_pages, table, lens, keep, 2, 5, 40) == 4


def test_select_pages_outside_the_pool(mla):
    lens = [300, 500]
    table, num_pages = tables(lens, 8, 13)
    table[0, 2], table[1, 0], table[1, 5] = -1, num_pages, 2 ** 31 - 1
    mass = weights(num_pages * 64, 14, "odd")
    for keep in ([60, 90], [290, 490]):
        assert check_select(mla, mass, num_pages, table, lens, keep, 0, 3, 500) == 2


def test_select_on_another_stream(mla):
    table, num_pages = tables([700, 800], 14, 15)
    check_select(mla, weights(num_pages * 64, 16, "spread"), num_pages, table, [700, 800], [70, 500], 4, 4, 500,
                 stream=torch.cuda.Stream())


# ---------------------------------------------------------------------------

def fill(mla, lf, kf, num_pages, seed):
    g = torch.Generator().manual_seed(seed)
    outl = sorted(torch.randperm(512, generator=g)[:25].tolist()) if lf == F_I8OUT else None
    cache = mla.CacheLayer(num_pages, lf, kf, outlier_channels=outl)
    cache.pool.copy_(torch.randint(0, 256, cache.pool.shape, dtype=torch.uint8, generator=g))     # any bits
    return cache


def expect_move(cache, lf, kf, src, lens, kept, new, dst, mass):
    """The pool's and masses' expected state, token by token through the documented layout."""
    L = cache.layout
    pool = cache.pool.cpu().numpy().copy()
    want = {}
    for b in range(len(lens)):
        if new[b] == lens[b]:
            continue
        slots_from = [int(src[b, t // 64]) * 64 + t % 64 for t in kept[b, :new[b]]]
        slots_to = [int(dst[b, j // 64]) * 64 + j % 64 for j in range(new[b])]
        want[b] = slots_to, read_tokens(pool, L, lf, kf, slots_from), mass[slots_from].copy()
    return want


@pytest.mark.parametrize("lf,kf", EVERY, ids=lambda f: FMT_NAME.get(f, str(f)))
def test_move_every_format(mla, lf, kf):
    lens = [200, 64, 1, 500, 130, 33]
    new = [70, 64, 0, 499, 1, 32]
    src, n1 = tables(lens, 8, 20)
    dst, num_pages = tables(new, 8, 21, first=n1)
    r = random.Random(22)
    width = 500
    kept = np.full((6, width), -1, np.int32)
    for b, (t, k) in enumerate(zip(lens, new)):
        kept[b, :k] = sorted(r.sample(range(t), k))
    cache = fill(mla, lf, kf, num_pages, 23)
    mass = torch.rand(num_pages * 64, generator=torch.Generator().manual_seed(24)).numpy()
    before = cache.pool.cpu().numpy().copy()
    want = expect_move(cache, lf, kf, src, lens, kept, new, dst, mass)
    d_mass, err = torch.from_numpy(mass.copy()).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_move_tokens(cache, dev(src), dev(lens), dev(kept), dev(new), dev(dst), mass=d_mass, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    after, got_mass = cache.pool.cpu().numpy(), d_mass.cpu().numpy()
    touched = np.zeros(num_pages * 64, bool)
    for b, (to, fields, m) in want.items():
        got = read_tokens(after, cache.layout, lf, kf, to)
        for k, v in fields.items():
            assert np.array_equal(got[k].view(np.uint8), v.view(np.uint8)), k       # bits: NaNs too
        assert np.array_equal(got_mass[to], m)
        touched[to] = True
    # every other slot is as it was
    rest = np.nonzero(~touched)[0]
    a, z = read_tokens(before, cache.layout, lf, kf, rest), read_tokens(after, cache.layout, lf, kf, rest)
    for k in a:
        assert np.array_equal(a[k].view(np.uint8), z[k].view(np.uint8)), k
    assert np.array_equal(got_mass[rest], mass[rest])


def test_move_without_mass_and_bad_figures(mla):
    lens, new = [200, 200, 200, 9 * 64, 200, 200], [50, 201, -1, 5, 60, 64]
    src, n1 = tables([200] * 6, 8, 30)
    dst, num_pages = tables([100] * 6, 8, 31, first=n1)
    kept = np.tile(np.arange(0, 200, 2, dtype=np.int32), (6, 1))
    kept[0, 3], kept[0, 5] = -1, 200                       # outside the sequence
    src[4, 1] = num_pages                                  # positions 64 .. 127 lie nowhere
    dst[5, 0] = -1
    cache = fill(mla, F_INT8, F_INT8, num_pages, 32)
    before = cache.pool.cpu().numpy().copy()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_move_tokens(cache, dev(src), dev(lens), dev(kept), dev(new), dev(dst), dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 1 | 2 | 4
    after = cache.pool.cpu().numpy()
    moved = {}
    for b in (0, 4):
        for j in range(new[b]):
            t = int(kept[b, j])
            if 0 <= t < 200 and not (b == 4 and t // 64 == 1):
                moved[int(dst[b, j // 64]) * 64 + j % 64] = int(src[b, t // 64]) * 64 + t % 64
    to = np.arange(num_pages * 64)
    came = np.array([moved.get(int(s), int(s)) for s in to])
    a, z = read_tokens(before, cache.layout, F_INT8, F_INT8, came), read_tokens(after, cache.layout, F_INT8, F_INT8, to)
    for k in a:
        assert np.array_equal(a[k].view(np.uint8), z[k].view(np.uint8)), k


def test_move_far_into_the_pool(mla):
    """Page offsets past 2^31 bytes."""
    num_pages = 50000                                      # 64 x 1152 bytes each: 3.7 GB
    cache = mla.CacheLayer(num_pages, F_BF16, F_BF16)
    src, dst = np.array([[num_pages - 1, 40000]], np.int32), np.array([[num_pages - 2, -1]], np.int32)
    L = cache.layout
    page = cache.pool.view(num_pages, L.page_bytes)
    page[num_pages - 1] = torch.randint(0, 256, (L.page_bytes,), dtype=torch.uint8, device="cuda")
    page[40000] = torch.randint(0, 256, (L.page_bytes,), dtype=torch.uint8, device="cuda")
    kept = np.array([list(range(1, 100, 2))], np.int32)
    mass = torch.arange(num_pages * 64, dtype=torch.float32, device="cuda")
    mla.mla_move_tokens(cache, dev(src), dev([100]), dev(kept), dev([50]), dev(dst), mass=mass)
    three = torch.stack([page[num_pages - 1], page[40000], page[num_pages - 2]]).cpu().numpy().reshape(-1)
    a = read_tokens(three, L, F_BF16, F_BF16, [t for t in kept[0]])
    z = read_tokens(three, L, F_BF16, F_BF16, [128 + j for j in range(50)])
    assert all(np.array_equal(a[k], z[k]) for k in a)
    assert mass[(num_pages - 2) * 64 + 40].item() == float(40000 * 64 + 81 - 64)
