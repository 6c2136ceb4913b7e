"""mla_chunk_attention on the GPU against the formula in 64 bits, over ragged
batches, formats, masks and the ways a program calls it."""

import math

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests import _step_reference as R
from tests._helpers import ALL_FORMATS, F_BF16, F_I8OUT, F_INT4, F_INT8, FMT_NAME

pytestmark = pytest.mark.gpu

NAN = float("nan")
RAGGED = [(0, 1), (63, 3), (5, 0), (200, 130), (64, 64), (1, 65), (300, 1), (0, 129)]     # (ctx, new) per sequence


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


class Batch:
    """A ragged batch with a filled cache.  Latents have uneven channels, some
    far from zero; scores spread over a few units."""

    def __init__(self, mla, lens, H, lf=F_INT8, kf=F_INT8, seed=0, spare=3, gain=1.0):
        g = torch.Generator().manual_seed(seed * 1000 + H + 7 * lf + kf)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.mla, self.H, self.B = mla, H, len(lens)
        self.ctx, self.new = [c for c, _ in lens], [n for _, n in lens]
        self.lens = [c + n for c, n in lens]
        self.N = sum(self.new)
        pages = [-(-t // 64) for t in self.lens]
        self.P = max(1, max(pages))
        self.num_pages = sum(pages) + spare
        ids = torch.randperm(self.num_pages, generator=g).tolist()
        self.table = torch.full((self.B, self.P), -1, dtype=torch.int32)
        for b, n in enumerate(pages):
            self.table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
        ch = torch.exp(0.6 * r(512))
        mean = 0.5 * r(512)
        self.c = [(mean + gain * ch * r(t, 512)).bfloat16() for t in self.lens]
        self.k = [r(t, 64).bfloat16() for t in self.lens]
        outl = None
        if lf == F_I8OUT:
            outl = sorted(torch.topk((mean.abs() + ch), 25).indices.tolist())
        self.cache = mla.CacheLayer(self.num_pages, lf, kf, outlier_channels=outl)
        self.cache.pool.fill_(0xFF)                     # unwritten tokens hold NaN patterns
        slots = [int(self.table[b, t // 64]) * 64 + t % 64 for b in range(self.B) for t in range(self.lens[b])]
        if slots:
            mla.mla_cache_append(self.cache, torch.cat(self.c).cuda(), torch.cat(self.k).cuda(),
                                 torch.tensor(slots, dtype=torch.int32, device="cuda"))
        self.hat = []
        for c, k in zip(self.c, self.k):
            if c.shape[0]:
                d = Q.quantize_token_rows(c.float().numpy(), k.float().numpy(), lf, kf, outliers=outl)
                self.hat.append((torch.from_numpy(np.asarray(d["c_hat"], np.float64)),
                                 torch.from_numpy(np.asarray(d["kpe_hat"], np.float64))))
            else:
                self.hat.append((torch.zeros(0, 512).double(), torch.zeros(0, 64).double()))
        self.q = r(self.N, H, 192).bfloat16()
        self.w_uk = (r(H, 128, 512) / math.sqrt(512)).bfloat16()
        self.w_uv = (r(H, 512, 128) / math.sqrt(512)).bfloat16()
        self.start = [sum(self.new[:b]) for b in range(self.B + 1)]
        self.dev = {k: getattr(self, k).cuda() for k in ("q", "w_uk", "w_uv", "table")}
        self.dev["start"] = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        self.dev["lens"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.max_new = max(self.new) if self.new else 0
        self.kv_tokens = sum(-(-t // 128) * 128 for t, n in zip(self.lens, self.new) if n > mla.CHUNK_SHORT)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, **kw):
        n = self.mla.mla_chunk_workspace_bytes(self.B, kw.get("N", self.N), self.H, kw.get("max_new", self.max_new),
                                               kw.get("kv_tokens", self.kv_tokens))
        assert n > 0
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")        # scratch that holds NaN patterns

    def call(self, ws=None, o=None, stream=None, **kw):
        N = kw.get("N", self.N)
        ws = self.workspace(**kw) if ws is None else ws
        o = torch.full((N, self.H, 128), NAN, dtype=torch.bfloat16, device="cuda") if o is None else o
        d = self.dev | kw.get("dev", {})
        self.mla.mla_chunk_attention(self.cache, d["q"][..., :128], d["q"][..., 128:], d["w_uk"], d["w_uv"], d["table"],
                                     d["start"], d["lens"], ws, o, max_new=kw.get("max_new", self.max_new),
                                     kv_tokens=kw.get("kv_tokens", self.kv_tokens), dev_err=self.err, stream=stream,
                                     softmax_scale=kw.get("scale"))
        return o

    def want(self, b, skip=None, scale=R.SCALE, heads=None):
        h = slice(None) if heads is None else heads
        c, k = self.hat[b]
        rows = slice(self.start[b], self.start[b + 1])
        q = self.q[rows, h].double()
        return R.chunk(c, k, q[..., :128], q[..., 128:], self.w_uk[h].double(), self.w_uv[h].double(), self.ctx[b],
                       scale=scale, skip=skip)

    def check(self, o, seqs=None, skip=None, scale=R.SCALE, heads=None):
        o = o.double().cpu() if heads is None else o[:, heads].double().cpu()
        off2 = mean2 = 0.0
        for b in range(self.B) if seqs is None else seqs:
            if not self.new[b]:
                continue
            want, bound, m2 = self.want(b, None if skip is None else skip.get(b), scale, heads)
            got = o[self.start[b]:self.start[b + 1]]
            d = (got - want).abs()
            assert not (~(d <= bound)).any(), "sequence %d: %g times the bound" % (b, float((d / bound).nan_to_num(1e9).max()))
            off2 += float((d ** 2).sum())
            mean2 += m2
        # thousands of independent roundings: their sum is near its mean; 1.5
        # covers the mean's own assumptions (errors spread evenly in a step)
        assert off2 <= 1.5 ** 2 * mean2, (off2 / mean2) ** 0.5


@pytest.mark.parametrize("lf,kf", ALL_FORMATS + [(F_I8OUT, F_BF16), (F_I8OUT, F_INT8)],
                         ids=lambda f: FMT_NAME.get(f, str(f)))
def test_every_format_over_a_ragged_batch(mla, lf, kf):
    t = Batch(mla, RAGGED, 16, lf, kf)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o)


@pytest.mark.parametrize("H", [32, 48, 64, 112, 128])
@pytest.mark.parametrize("lens", [[(70, 1), (0, 2)], [(130, 5), (3, 9), (0, 70)]], ids=["few", "more"])
def test_heads(mla, H, lens):
    t = Batch(mla, lens, H)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513])
@pytest.mark.parametrize("ctx", [0, 77])
def test_chunk_lengths(mla, n, ctx):
    t = Batch(mla, [(ctx, n)], 16, seed=n)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=slice(3, 7))


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 4095, 4096, 4097])
def test_context_lengths_of_a_single_token(mla, T):
    t = Batch(mla, [(T - 1, 1)], 16, F_INT4, F_INT8, seed=T)
    o = t.call()
    torch.cuda.synchronize()
    t.check(o)


@pytest.mark.parametrize("lf,kf", [(F_BF16, F_BF16), (F_INT8, F_INT8)], ids=["bf16", "int8"])
@pytest.mark.parametrize("lens", [[(20000, 1), (9000, 2), (13, 1)], [(9001, 200)]], ids=["decode", "chunk"])
def test_long_contexts(mla, lf, kf, lens):
    t = Batch(mla, lens, 16, lf, kf)
    o = t.call()
    torch.cuda.synchronize()
    t.check(o, heads=slice(0, 3))


def test_many_sequences(mla):
    r = np.random.default_rng(5)
    t = Batch(mla, [(int(r.integers(0, 150)), int(r.integers(0, 4))) for _ in range(400)], 16)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=slice(5, 7))


@pytest.mark.parametrize("B", [2, 30, 31, 151, 153, 310, 700])
@pytest.mark.parametrize("most", [64, 200])
def test_runs_that_end_between_sequences(mla, B, most):
    """Contexts of one to four pages: an SM's run ends before, at and behind
    a sequence's first page, and holds several sequences or none."""
    t = Batch(mla, [((37 * b + 11 * B) % most, 1 + (b % 5 == 3)) for b in range(B)], 16, seed=B)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o)


@pytest.mark.parametrize("B", [3, 9, 10, 38, 77])
@pytest.mark.parametrize("n", [65, 300])
def test_runs_that_end_between_chunks(mla, B, n):
    t = Batch(mla, [((53 * b) % 130, n - b % 2) for b in range(B)], 16, seed=B)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=[0, 7, 15])


def test_many_chunks(mla):
    r = np.random.default_rng(6)
    t = Batch(mla, [(int(r.integers(0, 300)), int(r.integers(60, 200))) for _ in range(12)], 16)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=slice(9, 11))


def test_rows_behind_the_last_sequence_stay(mla):
    t = Batch(mla, [(10, 3), (100, 70)], 16)
    q = torch.full((t.N + 13, 16, 192), NAN, dtype=torch.bfloat16, device="cuda")
    q[:t.N] = t.dev["q"]
    o = torch.full((t.N + 13, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    t.call(o=o, N=t.N + 13, dev={"q": q})
    torch.cuda.synchronize()
    assert t.err.item() == 0
    assert (o[t.N:] == 5).all()
    t.check(o[:t.N])


@pytest.mark.parametrize("big", [False, True], ids=["few", "chunk"])
def test_empty_and_refused_sequences(mla, big):
    """Length 0: zero rows, no flag.  Figures that do not fit: zero rows and
    the flag.  The neighbours are untouched."""
    n = 80 if big else 3
    t = Batch(mla, [(10, 2), (20, n), (30, n), (40, n), (50, 3)], 16)
    lens = t.dev["lens"].clone()
    lens[1] = 0
    o = t.call(dev={"lens": lens})
    torch.cuda.synchronize()
    assert t.err.item() == 0
    assert (o[t.start[1]:t.start[2]] == 0).all()
    t.check(o, seqs=[0, 2, 3, 4])
    for bad in (-5, n - 1, t.P * 64 + 1):
        lens[2] = bad
        o = t.call(dev={"lens": lens})
        torch.cuda.synchronize()
        assert t.err.item() == mla.DEVERR_SEQLEN
        t.err.zero_()
        assert (o[t.start[1]:t.start[3]] == 0).all()
        t.check(o, seqs=[0, 3, 4])


def test_more_new_tokens_than_announced(mla):
    t = Batch(mla, [(10, 2), (20, 9), (30, 4)], 16)
    o = t.call(max_new=4)
    torch.cuda.synchronize()
    assert t.err.item() == mla.DEVERR_SEQLEN
    assert (o[t.start[1]:t.start[2]] == 0).all()
    t.check(o, seqs=[0, 2])


def test_more_keys_than_announced(mla):
    """Chunks beyond kv_tokens are refused; the sequences before them and the
    short ones are computed."""
    t = Batch(mla, [(100, 70), (20, 9), (300, 80), (0, 1)], 16)
    o = t.call(kv_tokens=256)
    torch.cuda.synchronize()
    assert t.err.item() == mla.DEVERR_SEQLEN
    assert (o[t.start[2]:t.start[3]] == 0).all()
    t.check(o, seqs=[0, 1, 3])


def test_chunk_without_room_for_any(mla):
    """kv_tokens 0: chunks are refused, the decodes around them are served."""
    t = Batch(mla, [(70, 1), (10, 65), (200, 2)], 16)
    o = t.call(kv_tokens=0)
    torch.cuda.synchronize()
    assert t.err.item() == mla.DEVERR_SEQLEN
    assert not o[1:66].any()
    t.check(o, seqs=[0, 2])


@pytest.mark.parametrize("B", [127, 128, 129])
def test_batches_around_a_block_of_sequences(mla, B):
    t = Batch(mla, [((29 * b) % 100, (b + 1) % 3) for b in range(B)], 32, seed=B)
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=[3, 31])


def test_row_starts_out_of_order(mla):
    t = Batch(mla, [(10, 2), (20, 4), (30, 3)], 16)
    for start in ([0, 6, 2, 9], [-3, 2, 6, 9], [0, 2, 6, 900]):
        o = t.call(dev={"start": torch.tensor(start, dtype=torch.int32, device="cuda")})
        torch.cuda.synchronize()
        assert t.err.item() & mla.DEVERR_SEQLEN
        t.err.zero_()
    t.check(t.call())


@pytest.mark.parametrize("n", [1, 3, 90])
def test_pages_outside_the_pool(mla, n):
    """A page id outside the pool contributes nothing; a row that sees no
    other page is 0."""
    t = Batch(mla, [(200, n), (60, n), (5, n)], 16)
    table = t.dev["table"].clone()
    table[0, 1] = -1
    table[0, 2] = t.num_pages
    table[1, 0] = 2 ** 31 - 1
    o = t.call(dev={"table": table})
    torch.cuda.synchronize()
    assert t.err.item() == mla.DEVERR_PAGE
    s0, s1 = torch.zeros(t.lens[0], dtype=torch.bool), torch.zeros(t.lens[1], dtype=torch.bool)
    s0[64:192] = True
    s1[:64] = True
    t.check(o, skip={0: s0, 1: s1})


@pytest.mark.parametrize("lf,kf", [(F_BF16, F_BF16), (F_INT8, F_INT8), (F_INT4, F_INT8)], ids=["bf16", "int8", "int4"])
@pytest.mark.parametrize("n", [6, 90])
@pytest.mark.parametrize("what", ["c", "k"])
def test_non_finite_tokens_reach_only_the_rows_that_see_them(mla, lf, kf, n, what):
    t = Batch(mla, [(70, n), (20, n)], 16, lf, kf)
    t_bad = 70 + n // 2
    c, k = t.c[0][t_bad:t_bad + 1].clone(), t.k[0][t_bad:t_bad + 1].clone()
    (c if what == "c" else k)[0, 33] = float("inf") if what == "c" else NAN
    slot = int(t.table[0, t_bad // 64]) * 64 + t_bad % 64
    mla.mla_cache_append(t.cache, c.cuda(), k.cuda(), torch.tensor([slot], dtype=torch.int32, device="cuda"))
    o = t.call()
    torch.cuda.synchronize()
    got = o.double().cpu()
    want, bound, _ = t.want(0)
    first = t_bad - 70                                   # the first new token that sees it
    assert ((got[:first] - want[:first]).abs() <= bound[:first]).all()
    if lf == F_BF16 or what == "c":                      # INT8 k_pe of a NaN: the append's maximum skips it
        assert torch.isnan(got[first:n]).all()
    t.check(o, seqs=[1])


def test_non_finite_query_stays_in_its_row(mla):
    t = Batch(mla, [(70, 6), (20, 80)], 16)
    q = t.dev["q"].clone()
    q[2, 3, 5] = NAN
    q[50, 7, 150] = float("inf")
    o = t.call(dev={"q": q})
    torch.cuda.synchronize()
    assert torch.isnan(o[2, 3]).all() and torch.isnan(o[50, 7]).all()
    o[2, 3] = t.call()[2, 3]
    o[50, 7] = t.call()[50, 7]
    t.check(o)


@pytest.mark.parametrize("gain,scale", [(12.0, R.SCALE), (1.0, 1e-3), (1.0, 2.0)])
def test_peaked_and_flat_softmax(mla, gain, scale):
    t = Batch(mla, [(500, 4), (300, 70)], 16, F_BF16, F_BF16, gain=gain)
    o = t.call(scale=scale)
    torch.cuda.synchronize()
    got = o.double().cpu()
    for b in range(2):
        want, bound, _ = t.want(b, scale=scale, heads=slice(0, 4))
        assert ((got[t.start[b]:t.start[b + 1], :4] - want).abs() <= bound).all()


def test_strided_queries(mla):
    t = Batch(mla, [(70, 6), (20, 80)], 16)
    hm = t.dev["q"].transpose(0, 1).contiguous().transpose(0, 1)          # [H][N][192] in memory
    wide = torch.zeros((t.N, 16, 256), dtype=torch.bfloat16, device="cuda")
    wide[..., 32:224] = t.dev["q"]
    a, b, c = t.call(), t.call(dev={"q": hm}), t.call(dev={"q": wide[..., 32:224]})
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    t.check(a)


def test_repeats_are_identical(mla):
    t = Batch(mla, RAGGED, 16)
    ws = t.workspace()
    a = t.call(ws=ws)
    for _ in range(5):
        assert torch.equal(a, t.call(ws=ws))


def test_workspace_bounds(mla):
    """A workspace of exactly the stated size, with sentinels behind it."""
    t = Batch(mla, RAGGED, 16)
    n = mla.mla_chunk_workspace_bytes(t.B, t.N, t.H, t.max_new, t.kv_tokens)
    big = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    t.check(t.call(ws=big[:n]))
    assert (big[n:] == 0x5A).all()
    with pytest.raises(mla.MlaError):
        t.call(ws=big[:n - 1])


def test_two_streams_at_once(mla):
    a, b = Batch(mla, RAGGED, 16, seed=1), Batch(mla, [(900, 1)] * 20 + [(0, 100)], 16, seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = a.workspace(), b.workspace()
    oa, ob = a.call(ws=wa), b.call(ws=wb)
    torch.cuda.synchronize()
    pa, pb = torch.empty_like(oa), torch.empty_like(ob)
    torch.cuda.synchronize()
    for _ in range(10):
        a.call(ws=wa, o=pa, stream=s1)
        b.call(ws=wb, o=pb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(oa, pa) and torch.equal(ob, pb)
    a.check(pa, seqs=[1, 3])


def test_graph_replayed_with_other_lengths(mla):
    """One captured call, replayed as sequences grow and shrink: the bounds
    of the capture hold, the lengths are the device's."""
    t = Batch(mla, [(300, 80), (10, 4), (200, 90), (0, 1)], 16)
    cap = {"max_new": 120, "kv_tokens": 1024, "N": 256}
    q = torch.zeros((256, 16, 192), dtype=torch.bfloat16, device="cuda")
    start, lens = t.dev["start"].clone(), t.dev["lens"].clone()
    o = torch.full((256, 16, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = t.workspace(**cap)
    q[:t.N] = t.dev["q"]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t.call(ws=ws, o=o, dev={"q": q, "start": start, "lens": lens}, **cap)
    g.replay()
    torch.cuda.synchronize()
    t.check(o[:t.N])
    # the same cache read with fewer new tokens per sequence
    u = [(379, 1), (12, 2), (170, 120), (0, 1)]
    t.ctx, t.new = [c for c, _ in u], [n for _, n in u]
    t.lens = [c + n for c, n in u]
    t.hat = [(c[:n], k[:n]) for (c, k), n in zip(t.hat, t.lens)]
    t.start = [sum(t.new[:b]) for b in range(5)]
    t.q = torch.randn((t.start[4], 16, 192), generator=torch.Generator().manual_seed(9)).bfloat16()
    q[:t.start[4]] = t.q.cuda()
    start.copy_(torch.tensor(t.start, dtype=torch.int32))
    lens.copy_(torch.tensor(t.lens, dtype=torch.int32))
    o.fill_(5.0)
    g.replay()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    assert (o[t.start[4]:] == 5).all()
    t.check(o[:t.start[4]])


def test_pages_far_into_a_large_pool(mla):
    """Page offsets past 2^32 bytes."""
    t = Batch(mla, [(150, 2), (30, 70)], 16)
    lay = t.cache.layout
    far = (1 << 32) // lay.page_bytes + 50
    big = mla.CacheLayer(far + t.num_pages, F_INT8, F_INT8, pool=torch.empty((far + t.num_pages) * lay.page_bytes,
                                                                           dtype=torch.uint8, device="cuda"))
    big.pool[far * lay.page_bytes:] = t.cache.pool[:t.num_pages * lay.page_bytes]
    t.cache = big
    o = t.call(dev={"table": torch.where(t.dev["table"] >= 0, t.dev["table"] + far, t.dev["table"]).int()})
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o)


def test_agrees_with_the_decode_call(mla):
    """One new token per sequence: the decode's own output, within the two
    calls' bounds (the decode's 2e-3 of the row's largest latent output)."""
    t = Batch(mla, [(700, 1), (64, 1), (3, 1), (2000, 1)], 32)
    o = t.call()
    ql = torch.empty((4, 32, 512), device="cuda")
    mla.mla_q_absorb(t.dev["q"][..., :128].contiguous(), t.dev["w_uk"], ql)
    ws = torch.empty(mla.mla_decode_workspace_bytes(4, 32), dtype=torch.uint8, device="cuda")
    ol, o2 = torch.empty_like(ql), torch.empty((4, 32, 128), device="cuda")
    mla.mla_decode_absorbed_unabsorb(t.cache, ql, t.dev["q"][..., 128:].contiguous(), t.dev["table"], t.dev["lens"], ws,
                                     ol, t.dev["w_uv"], o2)
    torch.cuda.synchronize()
    t.check(o)
    for b in range(4):
        _, bound, _ = t.want(b)
        # sum_c 2e-3 max|o_lat| |W_UV| bounds the decode's share
        lat = 2e-3 * ol[b].abs().amax(-1, keepdim=True) * t.dev["w_uv"].abs().float().sum(1)
        assert ((o[b].float() - o2[b]).abs().cpu() <= bound[0].float() + lat.cpu()).all()


@pytest.mark.parametrize("lens", [[(900, 1)] * 5, [(300, 6), (20, 3)], [(700, 200)]], ids=["decode", "draft", "chunk"])
def test_waits_that_run_out_end_the_call(mla, lens):
    """With a wait limit of 0 the kernels give up, flag it and return; the
    next call, with the limit back, is whole."""
    t = Batch(mla, lens, 32)
    prev = mla.mla_set_wait_limit_ns(0)
    try:
        t.call()
        torch.cuda.synchronize()
    finally:
        mla.mla_set_wait_limit_ns(prev)
    assert t.err.item() == mla.DEVERR_TIMEOUT
    t.err.zero_()
    o = t.call()
    torch.cuda.synchronize()
    assert t.err.item() == 0
    t.check(o, heads=slice(30, 32))


def test_a_serving_step(mla):
    """plan -> rope -> append -> chunk attention over three steps of a small
    server (prefill chunks, then mixed, then decode), against the plain
    forms."""
    from tests.test_gpu_plan import call as plan_call, dev, outputs
    H, rows, P, num_pages = 16, 6, 8, 40
    g = torch.Generator().manual_seed(77)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w_uk, w_uv = (r(H, 128, 512) / 512 ** 0.5).bfloat16(), (r(H, 512, 128) / 512 ** 0.5).bfloat16()
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    cache = mla.CacheLayer(num_pages, F_INT8, F_INT8)
    cache.pool.fill_(0xFF)
    table = torch.full((rows, P), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(num_pages, generator=g).int().cuda()
    state = torch.tensor([0, num_pages], dtype=torch.int32, device="cuda")
    kept = {i: [] for i in range(rows)}                  # request -> [(latent, rotated key)], as appended
    ctx = [0] * rows
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for req, new in [([4, 1], [150, 70]), ([1, 0, 4, 5], [1, 90, 2, 0]), ([0, 4, 1], [1, 1, 1])]:
        n, B = sum(new) + 5, len(req)
        out = outputs(B, P, n)
        before = [ctx[i] for i in req]
        plan_call(mla, dev(before), dev(new), dev(req), table, free, state, num_pages, out, err)
        q, kv = r(n, H, 192).bfloat16().cuda(), r(n, 576).bfloat16().cuda()
        qo, ko = torch.empty((n, H, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 64), dtype=torch.bfloat16, device="cuda")
        mla.mla_rope(q[..., 128:], kv[:, 512:], out["positions"], freq.cuda(), qo, ko)
        mla.mla_cache_append(cache, kv[:, :512].contiguous(), ko, out["slot"], err)
        kvt = sum(-(-(c + m) // 128) * 128 for c, m in zip(before, new) if m > mla.CHUNK_SHORT)
        ws = torch.empty(mla.mla_chunk_workspace_bytes(B, n, H, max(new), kvt), dtype=torch.uint8, device="cuda")
        o = torch.full((n, H, 128), NAN, dtype=torch.bfloat16, device="cuda")
        mla.mla_chunk_attention(cache, q[..., :128], qo, w_uk.cuda(), w_uv.cuda(), out["block_table"], out["q_start"],
                                out["seq_lens"], ws, o, max_new=max(new), kv_tokens=kvt, dev_err=err)
        state[0:1] = out["free_head"]
        torch.cuda.synchronize()
        assert err.item() == 0
        assert torch.isnan(o[sum(new):]).all()
        row = 0
        for b, (i, m) in enumerate(zip(req, new)):
            pos = torch.arange(ctx[i], ctx[i] + m)
            sel = slice(row, row + m)
            # the rotation against its formula, then the attention on what it gave
            for x, y in ((q[sel, :, 128:], qo[sel]), (kv[sel, 512:], ko[sel])):
                x = x.double().cpu()
                want = R.rope(x, pos[None], freq, [0] * 32, True, False, 1.0)
                assert ((y.double().cpu() - want).abs() <= R.rope_bound(want, x, 1.0)).all()
            kept[i].append((kv[sel, :512].cpu(), ko[sel].cpu()))
            ctx[i] += m
            if m:
                d = Q.quantize_token_rows(torch.cat([a for a, _ in kept[i]]).float().numpy(),
                                          torch.cat([a for _, a in kept[i]]).float().numpy(), F_INT8, F_INT8)
                want, bound, _ = R.chunk(torch.from_numpy(np.asarray(d["c_hat"], np.float64)),
                                         torch.from_numpy(np.asarray(d["kpe_hat"], np.float64)),
                                         q[sel, :, :128].double().cpu(), qo[sel].double().cpu(), w_uk.double(),
                                         w_uv.double(), ctx[i] - m)
                assert ((o[sel].double().cpu() - want).abs() <= bound).all()
            row += m
