"""mla_token_mass on the GPU against the formula in 64 bits."""

import math

import numpy as np
import pytest
import torch

from tests import _stay_reference as R
from tests._helpers import ALL_FORMATS, F_BF16, F_I8OUT, F_INT4, F_INT4S, F_INT8, FMT_NAME
from tests.test_gpu_chunk import RAGGED, Batch

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


class Mass(Batch):
    """A batch with absorbed queries, the attention's log-sum-exp (in 64 bits,
    rounded once) and masses from before."""

    def __init__(self, mla, lens, H, lf=F_INT8, kf=F_INT8, seed=0, counted=None, decay=0.75, scale=SCALE, q_gain=0.5, **kw):
        super().__init__(mla, lens, H, lf, kf, seed, **kw)
        g = torch.Generator().manual_seed(seed + 99)
        self.q_lat = torch.randn((self.N, H, 512), generator=g) * q_gain
        self.q_pe = torch.randn((self.N, H, 64), generator=g).bfloat16()
        self.before = torch.rand(self.num_pages * 64, generator=g) + 0.5
        self.counted, self.decay, self.scale = counted, decay, scale
        self.lse = torch.zeros((self.N, H))
        for b in range(self.B):
            if self.new[b]:
                c, k = self.hat[b]
                rows = slice(self.start[b], self.start[b + 1])
                s = torch.einsum("nhc,tc->nht", torch.cat([self.q_lat[rows].double(), self.q_pe[rows].double()], -1), torch.cat([c, k], -1))
                seen = torch.ones((self.new[b], self.lens[b]), dtype=torch.bool).tril(self.ctx[b])[:, None, :]
                self.lse[rows] = torch.logsumexp((s * scale).masked_fill(~seen, -INF), -1).float()

    def go(self, mass=None, ws=None, stream=None, **kw):
        mass = self.before.cuda() if mass is None else mass
        n = self.mla.mla_mass_workspace_bytes(self.B, self.N, self.H, kw.get("max_new", self.max_new))
        assert n > 0
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        d = self.dev | kw.get("dev", {})
        counted = None if self.counted is None else torch.tensor(self.counted, dtype=torch.int32, device="cuda")
        args = self.q_lat.cuda(), self.q_pe.cuda(), self.lse.cuda()
        if stream is not None:
            torch.cuda.synchronize()
        self.mla.mla_token_mass(self.cache, *args, d["table"], d["start"], d["lens"], ws, mass, max_new=kw.get("max_new", self.max_new),
                                decay=self.decay, counted=counted, dev_err=self.err, softmax_scale=self.scale, stream=stream)
        torch.cuda.synchronize()
        return mass

    def compare(self, mass, alone=(), skip_pages=()):
        """alone: sequences that the call leaves alone."""
        got = mass.double().cpu()
        untouched = np.ones(self.num_pages * 64, bool)
        off2 = all2 = 0.0
        for b in range(self.B):
            if not self.new[b] or not self.lens[b] or b in alone:
                continue
            rows = slice(self.start[b], self.start[b + 1])
            want, bound = R.mass(*self.hat[b], self.q_lat[rows].double(), self.q_pe[rows].double(), self.lse[rows].double(),
                                 self.ctx[b], self.scale)
            t = np.arange(self.lens[b])
            slot = self.table[b].numpy()[t // 64].astype(np.int64) * 64 + t % 64
            ok = np.isin(t // 64, [p for s, p in skip_pages if s == b], invert=True)
            old = torch.where(torch.from_numpy(t) < (self.ctx[b] if self.counted is None else self.counted[b]),
                              self.before[torch.from_numpy(np.where(ok, slot, 0))].double() * float(np.float32(self.decay)), 0.0)
            d = (got[torch.from_numpy(np.where(ok, slot, 0))] - old - want).abs()
            # the old mass times decay, and the sum, are rounded once each
            lim = bound + 2.0 ** -23 * (old + want)
            assert not (~(d <= lim))[torch.from_numpy(ok)].any(), (b, float((d / lim)[torch.from_numpy(ok)].nan_to_num(1e9).max()))
            off2 += float((d[torch.from_numpy(ok)] ** 2).sum())
            all2 += float(((old + want)[torch.from_numpy(ok)] ** 2).sum())
            untouched[slot[ok]] = False
        # an fp32 result: well inside 1e-5 of the whole
        assert off2 <= (5e-6) ** 2 * all2 or all2 == 0, math.sqrt(off2 / all2)
        assert np.array_equal(got.numpy()[untouched], self.before.double().numpy()[untouched])


@pytest.mark.parametrize("lf,kf", ALL_FORMATS + [(F_I8OUT, F_BF16), (F_I8OUT, F_INT8)], ids=lambda f: FMT_NAME.get(f, str(f)))
def test_every_format_over_a_ragged_batch(mla, lf, kf):
    t = Mass(mla, RAGGED, 16, lf, kf)
    m = t.go()
    assert t.err.item() == 0
    t.compare(m)


@pytest.mark.parametrize("H", [16, 32, 48, 64, 80, 112, 128])
@pytest.mark.parametrize("lens", [[(70, 1), (0, 2)], [(130, 5), (3, 9), (0, 40)]], ids=["few", "more"])
def test_heads(mla, H, lens):
    t = Mass(mla, lens, H)
    m = t.go()
    assert t.err.item() == 0
    t.compare(m)


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("ctx", [0, 77])
def test_query_counts(mla, n, ctx):
    t = Mass(mla, [(ctx, n)], 16, seed=n)
    t.compare(t.go())
    assert t.err.item() == 0


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 1000])
@pytest.mark.parametrize("lf,kf", [(F_INT8, F_INT8), (F_BF16, F_BF16), (F_INT4, F_INT4S)], ids=["int8", "bf16", "int4"])
def test_context_lengths(mla, T, lf, kf):
    t = Mass(mla, [(T - 1, 1), (T + 1, 2)], 16, lf, kf, seed=T)
    t.compare(t.go())
    assert t.err.item() == 0


def test_long_context_many_rows(mla):
    t = Mass(mla, [(5000, 40), (30, 3)], 32, F_INT4, F_INT8, seed=2)
    t.compare(t.go())


def test_many_sequences(mla):
    t = Mass(mla, [(i % 90, 1 + i % 3) for i in range(300)], 16, seed=3)
    t.compare(t.go())
    assert t.err.item() == 0


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, 1.25])
def test_decay_and_counted(mla, decay):
    lens = [(100, 2), (64, 1), (0, 5), (300, 3)]
    for counted in (None, [0, 0, 0, 0], [102, 64, 3, 150]):
        t = Mass(mla, lens, 16, seed=4, decay=decay, counted=counted)
        t.compare(t.go())
        assert t.err.item() == 0


def test_stale_masses_of_new_tokens_are_not_read(mla):
    t = Mass(mla, [(100, 2), (0, 70)], 16, seed=5, decay=0.0)
    for b in range(2):
        for p in range(t.ctx[b], t.lens[b]):
            t.before[int(t.table[b, p // 64]) * 64 + p % 64] = NAN
    m = t.go()
    t.before = t.before.nan_to_num(0.0)
    # slots behind the last token keep what they had
    t.compare(m.nan_to_num(0.0))


def test_a_row_sums_to_one(mla):
    """Every row hands out a weight of 1 in all."""
    t = Mass(mla, [(700, 6)], 32, seed=6, counted=[0])
    m = t.go(mass=torch.zeros(t.num_pages * 64, device="cuda"))
    assert abs(float(m.double().sum()) - 6 * 32) < 6 * 32 * 1e-5


def test_with_the_decodes_own_lse(mla):
    """The lse of mla_decode_absorbed and mla_prefill_absorbed as they come (good to 2e-3)."""
    t = Mass(mla, [(600, 1), (90, 1), (1, 1)], 16, seed=7, counted=[0, 0, 0])
    ws = torch.empty(mla.mla_decode_workspace_bytes(3, 16), dtype=torch.uint8, device="cuda")
    lse, o = torch.empty((3, 16), device="cuda"), torch.empty((3, 16, 512), device="cuda")
    mla.mla_decode_absorbed(t.cache, t.q_lat.cuda(), t.q_pe.cuda(), t.dev["table"], t.dev["lens"], ws, o, lse)
    torch.cuda.synchronize()
    assert (lse.cpu() - t.lse).abs().max() < 2e-3
    t.lse = lse.cpu()
    t.compare(t.go())


@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_rows_without_a_finite_lse_add_nothing(mla, value):
    t = Mass(mla, [(100, 2), (40, 3)], 16, seed=8)
    t.lse[1, 3:9] = value
    t.lse[2] = value
    t.compare(t.go())


def test_garbage_behind_the_last_token(mla):
    """Unwritten slots of the last page hold NaN patterns (the batch's pool is
    filled with them): nothing of them is seen, in any format."""
    for lf, kf in ((F_INT8, F_INT8), (F_BF16, F_BF16), (F_INT4, F_INT4S), (F_I8OUT, F_BF16)):
        t = Mass(mla, [(0, 1), (32, 1), (95, 2)], 16, lf, kf, seed=9)
        t.compare(t.go())


def test_pages_outside_the_pool(mla):
    t = Mass(mla, [(300, 2), (200, 1)], 16, seed=10)
    table = t.table.clone()
    table[0, 1], table[0, 4], table[1, 2] = -1, t.num_pages, 2 ** 31 - 1
    m = t.go(dev={"table": table.cuda()})
    assert t.err.item() == 2
    t.compare(m, skip_pages=((0, 1), (0, 4), (1, 2)))


def test_figures_that_do_not_fit(mla):
    lens = [(100, 2), (50, 1), (30, 4), (64, 1), (9, 1)]
    t = Mass(mla, lens, 16, seed=11)
    bad = torch.tensor([102, -1, 3, t.P * 64 + 1, 10], dtype=torch.int32, device="cuda")
    m = t.go(dev={"lens": bad})
    assert t.err.item() == 4
    t.compare(m, alone=(1, 2, 3))
    t.err.zero_()
    t.compare(t.go(max_new=2), alone=(2,))
    assert t.err.item() == 4
    t.err.zero_()
    t.counted = [-1, 52, 10, 65, 10]
    t.compare(t.go(), alone=(0, 1))
    assert t.err.item() == 4
    for start in ([0, 2, 1, 7, 8, 9], [-1, 2, 3, 7, 8, 9], [0, 2, 3, 7, 8, 10]):
        t.err.zero_()
        m = t.go(dev={"start": torch.tensor(start, dtype=torch.int32, device="cuda")})
        assert t.err.item() == 4
        t.compare(m, alone=range(5))


def test_sequences_without_queries_or_tokens(mla):
    t = Mass(mla, [(100, 0), (0, 0), (20, 2)], 16, seed=12)
    t.compare(t.go())
    assert t.err.item() == 0


def test_a_window_of_the_latest_queries(mla):
    """Queries may be fewer than the step's tokens: all tokens before theirs start from 0 with counted = 0."""
    t = Mass(mla, [(968, 32), (480, 20)], 16, seed=13, counted=[0, 0])
    t.compare(t.go())


def test_tiny_and_large_values(mla):
    """Latents of 1e-3 against queries of 100, and the other way round."""
    for gain, q in ((1e-3, 100.0), (60.0, 0.01)):
        t = Mass(mla, [(150, 2)], 16, F_INT8, F_BF16, seed=14, gain=gain, scale=SCALE / 8, q_gain=q)
        t.compare(t.go())


def test_repeats_bit_for_bit(mla):
    t = Mass(mla, [(3000, 3), (100, 40), (0, 1)], 48, seed=16)
    a = t.go()
    for _ in range(3):
        assert torch.equal(a, t.go())


def test_in_a_graph_with_other_lengths(mla):
    t = Mass(mla, [(300, 2), (90, 2)], 16, seed=17)
    n = mla.mla_mass_workspace_bytes(2, 4, 16, 2)
    ws, mass = torch.empty(n, dtype=torch.uint8, device="cuda"), t.before.cuda()
    d = [t.q_lat.cuda(), t.q_pe.cuda(), t.lse.cuda()]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        mla.mla_token_mass(t.cache, *d, t.dev["table"], t.dev["start"], t.dev["lens"], ws, mass, max_new=2, decay=t.decay)
    g.replay()
    torch.cuda.synchronize()
    t.compare(mass)
    u = Mass(mla, [(200, 2), (10, 2)], 16, seed=18)
    u.table = torch.nn.functional.pad(u.table, (0, t.P - u.P), value=-1)
    u.cache, pool = t.cache, u.cache.pool
    t.cache.pool[: pool.numel()] = pool
    d[0].copy_(u.q_lat), d[1].copy_(u.q_pe), d[2].copy_(u.lse)
    t.dev["table"].copy_(u.table), t.dev["lens"].copy_(u.dev["lens"])
    mass[: u.before.numel()] = u.before.cuda()
    g.replay()
    torch.cuda.synchronize()
    u.compare(mass[: u.before.numel()])


@pytest.mark.parametrize("lf,kf", [(F_INT8, F_INT8), (F_BF16, F_BF16), (F_INT4, F_INT4S), (F_INT4S, F_INT8)], ids=lambda f: FMT_NAME[f])
def test_many_sequences_of_one_row_tile(mla, lf, kf):
    """Decodes of 16 heads: more sequences than SMs, lengths around pages and blocks."""
    lens = [(t, 1) for t in ([0, 1, 30, 31, 32, 33, 62, 63, 64, 65, 94, 95, 96, 127, 128, 129] * 14 + [2000, 700])]
    t = Mass(mla, lens, 16, lf, kf, seed=22)
    t.compare(t.go())
    assert t.err.item() == 0


def test_scales_and_zero_points_of_any_size(mla):
    """Groups whose values differ by little, far from zero (large zero-points), and groups of very different scale."""
    for lf, kf, gain in ((F_INT4, F_INT8, 1e-3), (F_INT4, F_INT4S, 30.0), (F_INT8, F_INT4S, 1e-4), (F_INT8, F_INT8, 100.0)):
        for H in (16, 32):
            t = Mass(mla, [(200, 1), (70, 1)], H, lf, kf, seed=23, gain=gain, scale=SCALE / max(1.0, gain), q_gain=0.3)
            t.compare(t.go())


def test_a_bound_above_the_step_s_figures(mla):
    """max_new larger than any sequence's: another kernel, the same masses."""
    t = Mass(mla, [(300, 1), (90, 1), (5, 1)], 16, seed=24)
    n = mla.mla_mass_workspace_bytes(t.B, t.N, 16, 3)
    t.compare(t.go(max_new=3, ws=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")))
    t.compare(t.go(max_new=1))


def test_two_calls_at_once(mla):
    """Two streams, a workspace each."""
    a, b = Mass(mla, [(3000, 2)], 16, seed=19), Mass(mla, [(2500, 5)], 32, F_INT4, F_INT8, seed=20)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [a.go(), b.go()]
    ws = [torch.empty(mla.mla_mass_workspace_bytes(1, t.N, t.H, t.max_new), dtype=torch.uint8, device="cuda") for t in (a, b)]
    put = [[t.q_lat.cuda(), t.q_pe.cuda(), t.lse.cuda()] for t in (a, b)]
    for _ in range(5):
        got = [t.before.cuda() for t in (a, b)]
        torch.cuda.synchronize()
        for t, st, w, x, m in zip((a, b), s, ws, put, got):
            mla.mla_token_mass(t.cache, *x, t.dev["table"], t.dev["start"], t.dev["lens"], w, m, max_new=t.max_new, decay=t.decay,
                               stream=st)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("H,lens", [(16, [(3000, 1), (500, 1)]), (32, [(3000, 1), (500, 1)]), (64, [(900, 5), (300, 4)])],
                         ids=["few rows", "resident", "streamed"])
def test_waits_that_run_out_end_the_call(mla, H, lens):
    """With no patience the kernel gives up and says so; the context stays usable and the next call is right."""
    t = Mass(mla, lens, H, seed=21)
    want = t.go()
    prev = mla.mla_set_wait_limit_ns(0)
    try:
        for _ in range(3):
            t.go()
    finally:
        mla.mla_set_wait_limit_ns(prev)
    assert t.err.item() in (0, mla.DEVERR_TIMEOUT)
    t.err.zero_()
    assert torch.equal(t.go(), want) and t.err.item() == 0


@pytest.mark.parametrize("lf,kf,H", [(F_BF16, F_BF16, 16), (F_INT8, F_INT8, 16), (F_INT8, F_BF16, 16), (F_BF16, F_BF16, 32),
                                     (F_INT4, F_INT8, 32), (F_INT8, F_INT8, 64), (F_INT8, F_BF16, 128)],
                         ids=lambda f: FMT_NAME.get(f, str(f)))
def test_hundreds_of_megabytes_of_pages(mla, lf, kf, H):
    """Long runs of key tiles from memory that no cache holds, ragged ends: copies
    land late and out of order.  The pages are copies of a few, so that 64 bits are soon
    done."""
    one = Batch(mla, [(639, 1)], H, lf, kf, seed=31, spare=0)
    B, P = 24, 250
    g = torch.Generator().manual_seed(32)
    pages = one.cache.pool.view(10, -1)
    perm, of = torch.randperm(B * P, generator=g).cuda(), torch.randint(0, 10, (B * P,), generator=g).cuda()
    pool = torch.empty((B * P, pages.shape[1]), dtype=torch.uint8, device="cuda")
    pool[perm] = pages[one.table[0].long().cuda()[of]]
    cache = mla.CacheLayer(B * P, lf, kf, pool=pool.view(-1))
    lens = [P * 64 - 301 * b for b in range(B)]
    q_lat, q_pe = torch.randn((B, H, 512), generator=g) * 0.5, torch.randn((B, H, 64), generator=g).bfloat16()
    lse = 6.0 + torch.randn((B, H), generator=g)
    ws = torch.empty(mla.mla_mass_workspace_bytes(B, B, H, 1), dtype=torch.uint8, device="cuda")
    args = [x.cuda() for x in (q_lat, q_pe, lse)] + [perm.int().view(B, P), torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                                                     torch.tensor(lens, dtype=torch.int32, device="cuda"), ws]
    want = [R.mass(*one.hat[0], q_lat[b:b + 1].double(), q_pe[b:b + 1].double(), lse[b:b + 1].double(), 639, SCALE) for b in range(B)]
    err, first = torch.zeros(1, dtype=torch.int32, device="cuda"), None
    for _ in range(12):
        mass = torch.full((B * P * 64,), 7.0, device="cuda")
        mla.mla_token_mass(cache, *args, mass, max_new=1, decay=0.0, dev_err=err, softmax_scale=SCALE)
        first = mass if first is None else first
        assert torch.equal(mass, first)
    assert err.item() == 0
    got = first.view(-1, 64)[perm].view(B, P * 64).double().cpu()
    src = (64 * of.view(B, P, 1) + torch.arange(64, device="cuda")).flatten(1).cpu()
    for b in range(B):
        w, bound = want[b][0][src[b]], want[b][1][src[b]]
        d = (got[b] - w).abs()[: lens[b]]
        assert bool((d <= (bound + 2.0 ** -23 * w)[: lens[b]]).all()), (b, float((d / bound[: lens[b]]).max()))
        assert bool((got[b, lens[b]:] == 7.0).all())
