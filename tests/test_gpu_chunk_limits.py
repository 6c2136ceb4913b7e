"""mla_chunk_attention at the edges of its ranges: many short segments, very
uneven weights, small scales, waits that run out anywhere."""

import time

import pytest
import torch

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
