"""mla_rope on the GPU against the formula in 64 bits."""

import pytest
import torch

from tests import _step_reference as R

pytestmark = pytest.mark.gpu

AXES = {1: [0] * 32, 2: [0, 1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12, 4: [0, 1, 2, 3] * 8}


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def inputs(n, H, axes, far, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * n + H)
    q = torch.randn((n, H, 192), generator=g).bfloat16().cuda()
    kv = torch.randn((n, 576), generator=g).bfloat16().cuda()
    pos = torch.randint(-far, far, (axes, n), generator=g, dtype=torch.int64).int().cuda()
    f = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    return q, kv, pos, f


def check(got, x, pos, f, axis, il, inv, amp):
    x, pos, f = x.double().cpu(), pos.cpu(), f.cpu()
    y = R.rope(x, pos, f, axis, il, inv, amp)
    bad = (got.double().cpu() - y).abs() > R.rope_bound(y, x, amp)
    assert not bad.any(), bad.nonzero()[:4]


@pytest.mark.parametrize("il", [True, False])
@pytest.mark.parametrize("inv", [False, True])
@pytest.mark.parametrize("n,H,axes,far,amp", [(1, 16, 1, 4096, 1.0), (7, 1, 2, 100, 0.7), (3, 128, 3, 1 << 20, 1.0),
                                              (65, 17, 4, 1 << 30, 1.3), (1000, 48, 3, 32768, 1.0), (5, 0, 1, 9, 1.0),
                                              (2500, 16, 1, 2 ** 31 - 1, -1.0)])
def test_matches_the_formula(mla, n, H, axes, far, amp, il, inv):
    q, kv, pos, f = inputs(n, H, axes, far)
    qo = torch.full((n, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = torch.full((n, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    mla.mla_rope(q[..., 128:], kv[:, 512:], pos, f, qo, ko, pair_axis=AXES[axes], interleaved=il, inverse=inv, amplitude=amp)
    torch.cuda.synchronize()
    check(qo, q[..., 128:], pos, f, AXES[axes], il, inv, amp)
    check(ko, kv[:, 512:], pos, f, AXES[axes], il, inv, amp)


@pytest.mark.parametrize("il", [True, False])
def test_in_place_on_slices_leaves_the_rest(mla, il):
    q, kv, pos, f = inputs(77, 16, 1, 5000)
    q0, kv0 = q.clone(), kv.clone()
    mla.mla_rope(q[..., 128:], kv[:, 512:], pos[0], f, q[..., 128:], kv[:, 512:], interleaved=il)
    torch.cuda.synchronize()
    assert torch.equal(q[..., :128], q0[..., :128]) and torch.equal(kv[:, :512], kv0[:, :512])
    check(q[..., 128:], q0[..., 128:], pos, f, AXES[1], il, False, 1.0)
    check(kv[:, 512:], kv0[:, 512:], pos, f, AXES[1], il, False, 1.0)


def test_keys_alone_queries_alone_and_head_major_layout(mla):
    q, kv, pos, f = inputs(50, 32, 1, 5000)
    hm = torch.empty((32, 50, 64), dtype=torch.bfloat16, device="cuda")
    mla.mla_rope(q[..., 128:], None, pos, f, hm.transpose(0, 1), None)
    torch.cuda.synchronize()
    check(hm.transpose(0, 1), q[..., 128:], pos, f, AXES[1], True, False, 1.0)


@pytest.mark.parametrize("il", [True, False])
def test_inverse_is_the_gradient(mla, il):
    """d/dx of <w, rope(x)> is the inverse applied to w: against differences
    of the 64-bit form along random directions, and the two calls' product."""
    n, H = 9, 16
    q, kv, pos, f = inputs(n, H, 3, 3000)
    w = torch.randn((n, H, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    gw = torch.empty_like(w)
    mla.mla_rope(w, None, pos, f, gw, None, pair_axis=AXES[3], interleaved=il, inverse=True, amplitude=1.25)
    torch.cuda.synchronize()
    x, wd = q[..., 128:].double().cpu(), w.double().cpu()
    for k in range(4):
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(k), dtype=torch.float64)
        e = 1e-4
        hi, lo = (R.rope(x + s * e * d, pos.cpu(), f.cpu(), AXES[3], il, False, 1.25) for s in (1, -1))
        num = float((wd * (hi - lo) / (2 * e)).sum())
        got = float((gw.double().cpu() * d).sum())
        # each of gw's values is off by its bound at most
        tol = float((R.rope_bound(gw.double().cpu(), wd, 1.25) * d.abs()).sum()) + 1e-6 * abs(num)
        assert abs(num - got) <= tol


def test_graph_replay_and_another_stream(mla):
    q, kv, pos, f = inputs(20, 16, 1, 5000)
    qo, ko = torch.empty((20, 16, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((20, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mla.mla_rope(q[..., 128:], kv[:, 512:], pos, f, qo, ko)
    pos += 17
    g.replay()
    torch.cuda.synchronize()
    check(qo, q[..., 128:], pos, f, AXES[1], True, False, 1.0)
    s = torch.cuda.Stream()
    qo2, ko2 = torch.empty_like(qo), torch.empty_like(ko)
    torch.cuda.synchronize()
    mla.mla_rope(q[..., 128:], kv[:, 512:], pos, f, qo2, ko2, stream=s)
    s.synchronize()
    assert torch.equal(qo, qo2) and torch.equal(ko, ko2)


def test_large_offsets(mla):
    """Rows more than 2^31 elements apart."""
    stride = (1 << 31) // 2 + 8
    base = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (3, 1, 64), (stride, 64, 1))
    x.copy_(torch.randn((3, 1, 64), generator=torch.Generator().manual_seed(4)).bfloat16())
    f = inputs(3, 1, 1, 9)[3]
    pos = torch.tensor([3, 400, 70000], dtype=torch.int32, device="cuda")
    out = torch.empty((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    mla.mla_rope(x, None, pos, f, out, None)
    torch.cuda.synchronize()
    check(out, x, pos[None], f, AXES[1], True, False, 1.0)
