"""mla_chunk_attention at the edges of its ranges: many short segments, very
uneven weights, small scales, waits that run out anywhere."""

import time

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests._helpers import F_BF16, F_INT8
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


def dominated(mla, B, H, n, T, x):  # noqa: F811
    """B sequences of n new tokens over the same T cached ones: the first key
    outweighs each of the others, which are nearly equal, by 128 x / sqrt(192)
    nats, and its latent is near zero.  Their weights add up to e^-17 T or so
    of the total, and all of the output comes from them."""
    t = Batch(mla, [(T - n, n)], H, F_BF16, F_BF16)
    g = torch.Generator().manual_seed(B + n)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    c, k = (1 + 0.1 * r(T, 512)).bfloat16(), (0.01 * r(T, 64)).bfloat16()
    c[0], k[0] = (1e-3 * r(512)).bfloat16(), x
    slots = (t.table[0].long()[:, None] * 64 + torch.arange(64)).reshape(-1)[:T].int()
    mla.mla_cache_append(t.cache, c.cuda(), k.cuda(), slots.cuda())
    q = torch.cat([0.01 * r(n, H, 128), torch.full((n, H, 64), 2.0)], -1).bfloat16()
    t.hat, t.q = [(c.double(), k.double())] * B, torch.cat([q] * B)
    t.B, t.N, t.new, t.ctx, t.lens = B, B * n, [n] * B, [T - n] * B, [T] * B
    t.start, t.kv_tokens = [n * b for b in range(B + 1)], (-(-T // 128) * 128 * B if n > mla.CHUNK_SHORT else 0)
    t.dev["q"], t.dev["table"] = t.q.cuda(), t.table.repeat(B, 1).cuda()
    t.dev["start"] = torch.tensor(t.start, dtype=torch.int32, device="cuda")
    t.dev["lens"] = torch.tensor(t.lens, dtype=torch.int32, device="cuda")
    return t


@pytest.mark.parametrize("x", [1.625, 1.75, 1.8671875, 1.9375], ids=["15.0", "16.2", "17.3", "17.9"])
@pytest.mark.parametrize("B,H,n", [(304, 16, 1), (304, 16, 2), (64, 16, 13), (1, 128, 80)], ids=["16", "32", "64", "long"])
def test_one_key_outweighs_thousands(mla, B, H, n, x):  # noqa: F811
    """Small weights keep their share however far below the largest one they
    are.  (So many sequences or heads that a block walks most of a context by
    itself.)"""
    t = dominated(mla, B, H, n, 65537, x)
    o = t.call().double().cpu()
    assert t.err.item() == 0
    want, bound, _ = t.want(0, heads=slice(0, 2))
    for b in {0, B // 2, B - 1}:
        d = (o[t.start[b]:t.start[b + 1], :2] - want).abs()
        assert (d <= bound).all(), "%g times the bound, %g of the output" % ((d / bound).max(), d.norm() / want.norm())


def test_small_scales_are_dequantized_with_one_rounding(mla):  # noqa: F811
    """The value code x scale of INT8 groups with scales from 2^-13 to 2^-7, as
    the attention holds it in fp16.  A sequence of one token gives its latents
    back, o = c W_UV.  Group 0 holds the values; groups 1 to 4 hold, in codes
    of a power-of-two scale u (which fp16 holds exactly), each value to within u
    2^-8 as two digits, and W_UV takes their difference: what is left is small,
    so that o's rounding to bf16 (2^-8 of it) does not hide fp16's.

    Bound, in half steps of fp16 at the value: 1 for the rounding, 1/8 for a
    scale rounded to 15 bits (2^-15 of a value below two steps of 2^11), with
    fp32 noise 2^-10."""
    B, H = 2000, 16
    r = np.random.default_rng(3)
    c = np.zeros((B, 512), np.float32)
    s0 = 2.0 ** -13 * 2.0 ** (6 * r.random(B))
    c[:, :16] = (r.integers(8, 128, (B, 16)) * r.choice([-1, 1], (B, 16))) * s0[:, None]
    c[:, 0] = 127 * s0
    c = torch.from_numpy(c).bfloat16().float().numpy()
    code, scale = Q.quantize_sym_int8(c[:, :16], 16)
    exact = code.astype(np.float64) * scale.astype(np.float64)
    u = 2.0 ** np.ceil(np.log2(scale.astype(np.float64)))         # [B, 1]
    hi = np.rint(exact / u)
    lo = np.rint((exact - hi * u) / (u / 128))
    assert np.abs(hi).max() <= 127 and np.abs(lo).max() <= 64
    w_uv = torch.zeros((H, 512, 128))
    for j in range(16):
        chans = [16 * (1 + j // 4) + 2 * (j % 4) + 1, 16 * (1 + j // 4) + 2 * (j % 4) + 2]
        c[:, chans[0]], c[:, chans[1]] = hi[:, j] * u[:, 0], lo[:, j] * u[:, 0]
        w_uv[:, j, j], w_uv[:, chans[0], j], w_uv[:, chans[1], j] = 1, -1, -1 / 128
    for g in range(1, 5):
        c[:, 16 * g] = 127 * u[:, 0]                              # makes the group's scale u
    x = torch.from_numpy(c).bfloat16()
    assert (x.float().numpy() == c).all()
    cache = mla.CacheLayer(B, F_INT8, F_INT8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    mla.mla_cache_append(cache, x.cuda(), torch.zeros((B, 64), dtype=torch.bfloat16, device="cuda"), i32(range(0, 64 * B, 64)))
    q = torch.zeros((B, H, 192), dtype=torch.bfloat16, device="cuda")
    o = torch.empty((B, H, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mla.mla_chunk_workspace_bytes(B, B, H, 1), dtype=torch.uint8, device="cuda")
    mla.mla_chunk_attention(cache, q[..., :128], q[..., 128:], torch.zeros((H, 128, 512), dtype=torch.bfloat16, device="cuda"),
                            w_uv.bfloat16().cuda(), i32(range(B)).view(B, 1), i32(range(B + 1)), i32([1] * B), ws, o, max_new=1)
    left = o[:, 0, :16].double().cpu().numpy()
    got = hi * u + lo * u / 128 + left
    half = 2.0 ** (np.floor(np.log2(np.abs(exact))) - 11)
    off = np.abs(got - exact) - 2.0 ** -8 * np.abs(left)
    worst = (off / half).max()
    assert worst <= 1 + 1 / 8 + 2.0 ** -10, worst


@pytest.mark.parametrize("limit", [0, 1000, 5000, 50000])
@pytest.mark.parametrize("lens", [[(40, 1)] * 3, [(0, 65)], [(300, 70), (20, 3)]], ids=["decode", "chunk", "both"])
def test_a_wait_that_runs_out_is_never_silent(mla, lens, limit):  # noqa: F811
    """Limits near the time that the waits take: whichever of them runs out, in
    whichever thread, a call either sets the flag or gives the whole result."""
    t = Batch(mla, lens, 16)
    ws = t.workspace()
    good = t.call(ws=ws)
    for _ in range(20):
        prev = mla.mla_set_wait_limit_ns(limit)
        try:
            o = t.call(ws=ws)
            torch.cuda.synchronize()
        finally:
            mla.mla_set_wait_limit_ns(prev)
        assert t.err.item() in (0, mla.DEVERR_TIMEOUT)
        assert t.err.item() or torch.equal(o, good)
        t.err.zero_()
    assert torch.equal(t.call(ws=ws), good)
    assert t.err.item() == 0


@pytest.mark.parametrize("length", [2 ** 31 - 64, 2 ** 31 - 127, 2 ** 31 - 128, 2 ** 24])
def test_a_chunk_of_a_length_near_32_bits_is_refused(mla, length):  # noqa: F811
    """A table of 2^25 - 1 pages allows lengths up to 2^31 - 64: a chunk that
    says so goes far past kv_tokens, and its neighbours are served."""
    t = Batch(mla, [(70, 2), (20, 90), (5, 1)], 16)
    table = torch.full((3, 2 ** 25 - 1), -1, dtype=torch.int32, device="cuda")
    table[:, :t.P] = t.dev["table"]
    lens = t.dev["lens"].clone()
    lens[1] = length
    o = t.call(dev={"table": table, "lens": lens})
    assert t.err.item() == mla.DEVERR_SEQLEN
    assert (o[t.start[1]:t.start[2]] == 0).all()
    t.check(o, seqs=[0, 2])
