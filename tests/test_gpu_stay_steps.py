"""Where the attention weight's log-sum-exps come from, positions after a cut,
and whole steps in a captured graph whose lengths live on the device."""

import random

import numpy as np
import pytest
import torch

from tests import _step_reference as S
from tests._helpers import F_BF16, F_INT4, F_INT8, FMT_NAME
from tests.test_gpu_mass import SCALE, Mass
from tests.test_gpu_stay_run import dev, e

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def queries_as_sequences(mla, t):
    """The lse of a ragged batch from one decode whose sequences are the
    queries: each its sequence's pages and the tokens that it sees."""
    of = torch.tensor([b for b in range(t.B) for _ in range(t.new[b])])
    seen = torch.tensor([t.ctx[b] + i + 1 for b in range(t.B) for i in range(t.new[b])], dtype=torch.int32)
    ws = torch.empty(mla.mla_decode_workspace_bytes(t.N, t.H), dtype=torch.uint8, device="cuda")
    lse, o = torch.empty((t.N, t.H), device="cuda"), torch.empty((t.N, t.H, 512), device="cuda")
    args = t.q_lat.cuda(), t.q_pe.cuda(), t.table[of].cuda(), seen.cuda()
    torch.cuda.synchronize()                              # the decode reads the lengths during the launch overlap
    mla.mla_decode_absorbed(t.cache, *args, ws, o, lse, t.err)
    return lse.cpu()


def prefill_by_sequence(mla, t):
    lse = torch.empty((t.N, t.H), device="cuda")
    for b in range(t.B):
        n, rows = t.new[b], slice(t.start[b], t.start[b + 1])
        if not n:
            continue
        ws = torch.empty(mla.mla_prefill_workspace_bytes(n, t.H), dtype=torch.uint8, device="cuda")
        o = torch.empty((n, t.H, 512), device="cuda")
        mla.mla_prefill_absorbed(t.cache, t.q_lat[rows].cuda(), t.q_pe[rows].cuda(), t.table[b].cuda(), t.ctx[b], ws, o, lse[rows], t.err)
    return lse.cpu()


@pytest.mark.parametrize("lf,kf", [(F_INT8, F_INT8), (F_BF16, F_BF16), (F_INT4, F_INT8)], ids=lambda f: FMT_NAME[f])
@pytest.mark.parametrize("lens", [[(600, 5), (90, 1), (0, 3), (300, 0), (1200, 4)], [(900, 40), (64, 64), (700, 32)]],
                         ids=["drafts", "windows"])
@pytest.mark.parametrize("source", [queries_as_sequences, prefill_by_sequence], ids=["decode", "prefill"])
def test_masses_from_the_librarys_own_lse(mla, source, lens, lf, kf):
    """Drafts and windows, from the decode and from the prefill: the lse is good
    to their documented 2e-3, and the masses are the formula's with it."""
    t = Mass(mla, lens, 16, lf, kf, seed=41, counted=[0] * len(lens))
    lse = source(mla, t)
    assert t.err.item() == 0 and (lse - t.lse).abs().max() < 2e-3
    t.lse = lse
    t.compare(t.go())
    # every row hands out a weight of 1 in all, to what the lse is off
    for b in range(t.B):
        slot = [int(t.table[b, p // 64]) * 64 + p % 64 for p in range(t.lens[b])]
        t.before.zero_()
        if t.new[b]:
            assert abs(float(t.go(mass=torch.zeros_like(t.before).cuda()).double().cpu()[slot].sum()) / (t.new[b] * 16) - 1) < 2.1e-3


def test_positions_after_a_cut(mla):
    """Kept tokens keep the rotation of their old positions.  The plan counts on
    from the shortened cache, so a program adds what a request lost."""
    B, P, H, num_pages, budget = 2, 8, 16, 40, 64
    g, r = torch.Generator().manual_seed(42), random.Random(43)
    inv_freq = 1.0 / 10000.0 ** (torch.arange(32) / 32.0)
    cache, mass = mla.CacheLayer(num_pages, F_BF16, F_BF16), torch.zeros(num_pages * 64, device="cuda")
    page_table, free, rng = torch.full((B, P), -1, dtype=torch.int32, device="cuda"), dev(list(range(num_pages))), dev([0, num_pages])
    req, ctx, lost, err = dev([1, 0]), dev([0] * B), dev([0] * B), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows, text = [[] for _ in range(B)], [0] * B           # (c, k before the rotation, position) of every cached token; the text's length
    ws = torch.empty(mla.mla_decode_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
    told = 0.0
    for step in range(7):
        new = [r.randint(60, 150) for _ in range(B)] if step == 0 else [r.randint(1, 40) for _ in range(B)]
        n = sum(new)
        table, start, lens, pos, who, slot, head = e(B, P), e(B + 1), e(B), e(n), e(n), e(n), e(1)
        mla.mla_plan_chunks(ctx, dev(new), req, page_table, free, rng, num_pages, table, start, lens, pos, who, slot, head, dev_err=err)
        rng = torch.stack([head[0], rng[1]])
        pos += lost[who.long()]
        want = [text[b] + i for b in range(B) for i in range(new[b])]
        assert pos.tolist() == want
        c, k = torch.randn((n, 512), generator=g).bfloat16(), torch.randn((n, 64), generator=g).bfloat16()
        q_pe = (2 * torch.randn((n, H, 64), generator=g)).bfloat16()
        q_out, k_out = torch.empty((n, H, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 64), dtype=torch.bfloat16, device="cuda")
        mla.mla_rope(q_pe.cuda(), k.cuda(), pos, inv_freq.cuda(), q_out, k_out)
        mla.mla_cache_append(cache, c.cuda(), k_out, slot, dev_err=err)
        at = 0
        for b in range(B):
            rows[b] += [(c[at + i].double(), k[at + i].double(), text[b] + i) for i in range(new[b])]
            at += new[b]
            text[b] += new[b]
        # the last token's attention over what is cached
        last = start[1:].long() - 1
        q_lat = 0.05 * torch.randn((B, H, 512), generator=g)
        o, lse = torch.empty((B, H, 512), device="cuda"), torch.empty((B, H), device="cuda")
        torch.cuda.synchronize()
        mla.mla_decode_absorbed(cache, q_lat.cuda(), q_out[last].contiguous(), table, lens, ws, o, lse, err)
        lse = lse.double().cpu()
        for b in range(B):
            x, y = torch.stack([a for a, _, _ in rows[b]]), torch.stack([a for _, a, _ in rows[b]])
            q = q_pe[int(last[b])].double()

            def scores(places, own):
                kr = S.rope(y, torch.tensor([places]), inv_freq, [0] * 32, True, False, 1.0)
                qr = S.rope(q, torch.tensor([[own] * H]), inv_freq, [0] * 32, True, False, 1.0)
                return (q_lat[b].double() @ x.t() + qr @ kr.t()) * SCALE, qr, kr

            s, qr, kr = scores([p for _, _, p in rows[b]], text[b] - 1)
            bq, bk = S.rope_bound(qr, q, 1.0), S.rope_bound(kr, y, 1.0)
            off = (((qr.abs() + bq) @ bk.t() + bq @ kr.abs().t()) * SCALE).amax(-1)
            assert ((lse[b] - torch.logsumexp(s, -1)).abs() <= off + 2e-3).all()
            # positions counted on from the shortened cache would be noticed
            wrong, _, _ = scores([p for _, _, p in rows[b]], len(rows[b]) - 1)
            told = max(told, float(((torch.logsumexp(wrong, -1) - torch.logsumexp(s, -1)).abs() / (off + 2e-3)).max()))
        ctx = lens
        if step % 2:
            continue
        mass.copy_(torch.rand(num_pages * 64, generator=g))
        kept, kept_lens, out, left, new_range = e(B, budget), e(B), e(B, P), e(B), e(2)
        mla.mla_select_tokens(mass, table, lens, dev([budget] * B), kept, kept_lens, sinks=2, recent=8, dev_err=err)
        mla.mla_release_pages(lens, kept_lens, req, table, page_table, free, rng, num_pages, out, left, new_range, move=True, dev_err=err)
        mla.mla_move_tokens(cache, table, lens, kept, left, out, mass=mass, dev_err=err)
        lost += lens - left
        ctx, rng = left, new_range
        for b in range(B):
            if len(rows[b]) > budget:
                rows[b] = [rows[b][i] for i in kept[b].tolist()]
    assert err.item() == 0 and told > 2.0


@pytest.mark.parametrize("lf,kf", [(F_INT8, F_INT8), (F_INT4, F_INT8)], ids=lambda f: FMT_NAME[f])
def test_whole_steps_in_a_graph(mla, lf, kf):
    """Plan, append, attention, attention weight, selection, release and move
    captured once; every replay goes on from the lengths that the one before
    left.  A copy of the lengths is the ordering point in front of the decode,
    which reads them during the launch overlap.  Against the same calls one by
    one, each waited for."""
    B, P, H, num_pages, budget = 3, 6, 16, 60, 100
    g = torch.Generator().manual_seed(44)
    new = dev([1, 2, 1])
    n, cap = 4, 5                                         # rows in use; the last has no token

    def state():
        cache = mla.CacheLayer(num_pages, lf, kf)
        cache.pool.zero_()
        return dict(cache=cache, mass=torch.zeros(num_pages * 64, device="cuda"), free=dev(list(range(num_pages))),
                    page_table=torch.full((B, P), -1, dtype=torch.int32, device="cuda"), rng=dev([0, num_pages]), ctx=dev([0] * B),
                    keep=dev([budget, budget - 3, budget + 40]), table=e(B, P), start=e(B + 1), lens=e(B), pos=e(cap), who=e(cap),
                    slot=e(cap), head=e(1), mid=e(2), seen=e(B), c=torch.zeros((cap, 512), dtype=torch.bfloat16, device="cuda"),
                    k=torch.zeros((cap, 64), dtype=torch.bfloat16, device="cuda"), q_lat=torch.zeros((B, H, 512), device="cuda"),
                    q_pe=torch.zeros((B, H, 64), dtype=torch.bfloat16, device="cuda"), o=torch.zeros((B, H, 512), device="cuda"),
                    lse=torch.zeros((B, H), device="cuda"), kept=e(B, budget + 40), kept_lens=e(B), out=e(B, P), left=e(B), after=e(2),
                    q_start=dev([0, 1, 2, 3]), err=torch.zeros(1, dtype=torch.int32, device="cuda"),
                    dws=torch.empty(mla.mla_decode_workspace_bytes(B, H), dtype=torch.uint8, device="cuda"),
                    ws=torch.empty(mla.mla_mass_workspace_bytes(B, B, H, 1), dtype=torch.uint8, device="cuda"))

    req = dev([2, 0, 1])

    def step(s, new, between):
        err = s["err"]
        mla.mla_plan_chunks(s["ctx"], new, req, s["page_table"], s["free"], s["rng"], num_pages, s["table"], s["start"], s["lens"],
                            s["pos"], s["who"], s["slot"], s["head"], dev_err=err)
        between()
        mla.mla_cache_append(s["cache"], s["c"], s["k"], s["slot"], dev_err=err)
        s["seen"].copy_(s["lens"])                        # a memory copy: a full ordering point
        between()
        mla.mla_decode_absorbed(s["cache"], s["q_lat"], s["q_pe"], s["table"], s["seen"], s["dws"], s["o"], s["lse"], err)
        between()
        mla.mla_token_mass(s["cache"], s["q_lat"], s["q_pe"], s["lse"], s["table"], s["q_start"], s["lens"], s["ws"], s["mass"], max_new=1,
                           decay=0.9, counted=s["ctx"], dev_err=err)
        between()
        mla.mla_select_tokens(s["mass"], s["table"], s["lens"], s["keep"], s["kept"], s["kept_lens"], sinks=2, recent=9, dev_err=err)
        s["mid"][:1].copy_(s["head"])
        s["mid"][1:].copy_(s["rng"][1:])
        between()
        mla.mla_release_pages(s["lens"], s["kept_lens"], req, s["table"], s["page_table"], s["free"], s["mid"], num_pages, s["out"],
                              s["left"], s["after"], move=True, dev_err=err)
        between()
        mla.mla_move_tokens(s["cache"], s["table"], s["lens"], s["kept"], s["left"], s["out"], mass=s["mass"], dev_err=err)
        s["ctx"].copy_(s["left"])
        s["rng"].copy_(s["after"])
        between()

    a, b = state(), state()
    prompt, more = dev([99, 97, 130]), 326
    c, k = torch.randn((more, 512), generator=g).bfloat16().cuda(), torch.randn((more, 64), generator=g).bfloat16().cuda()
    for s in (a, b):                                      # the prompts; this also loads the kernels before the capture
        wide = s | dict(pos=e(more), who=e(more), slot=e(more), c=c, k=k)
        step(wide, prompt, torch.cuda.synchronize)
        assert s["err"].item() == 0 and s["ctx"].tolist() == [99, 97, 130]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(a, new, lambda: None)
    cuts = 0
    for turn in range(20):
        for name in ("c", "k", "q_lat", "q_pe"):
            x = torch.randn(a[name].shape, generator=g).to(a[name].dtype)
            a[name].copy_(x)
            b[name].copy_(x)
        if turn == 12:
            for s in (a, b):
                s["keep"].copy_(dev([60, 140, 70]))
        before = b["ctx"].tolist()
        torch.cuda.synchronize()
        graph.replay()
        step(b, new, torch.cuda.synchronize)
        torch.cuda.synchronize()
        cuts += any(x < y for x, y in zip(b["ctx"].tolist(), before)) or b["left"].tolist() != b["lens"].tolist()
        for name in ("ctx", "rng", "page_table", "free", "table", "kept", "kept_lens", "out", "lse", "mass", "err"):
            assert torch.equal(a[name], b[name]), (turn, name)
        assert torch.equal(a["cache"].pool, b["cache"].pool), turn
    assert a["err"].item() == 0 and cuts >= 10 and n == int(new.sum())


def test_speculative_steps_in_a_graph(mla):
    """Plan, verification and trim captured once, the lengths handed on on the device."""
    B, P, V, num_pages, width = 3, 5, 400, 20, 4
    g = torch.Generator().manual_seed(45)
    req, new, rows = dev([1, 2, 0]), dev([4, 1, 3]), 8

    def state():
        return dict(free=dev(list(range(num_pages))), page_table=torch.full((B, P), -1, dtype=torch.int32, device="cuda"),
                    rng=dev([0, num_pages]), ctx=dev([40, 61, 126]), table=e(B, P), start=e(B + 1), lens=e(B), pos=e(rows), who=e(rows),
                    slot=e(rows), head=e(1), mid=e(2), p=torch.zeros((rows, V), device="cuda"), q=torch.zeros((rows, V), device="cuda"),
                    d=dev([0] * rows), ua=torch.zeros(rows, device="cuda"), us=torch.zeros(B, device="cuda"), acc=e(B), tok=e(B, width),
                    out=e(B, P), left=e(B), after=e(2), err=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def step(s, between):
        mla.mla_plan_chunks(s["ctx"], new, req, s["page_table"], s["free"], s["rng"], num_pages, s["table"], s["start"], s["lens"],
                            s["pos"], s["who"], s["slot"], s["head"], dev_err=s["err"])
        between()
        s["mid"][:1].copy_(s["head"])
        s["mid"][1:].copy_(s["rng"][1:])
        s["ctx"].copy_(s["lens"])
        mla.mla_verify_drafts(s["p"], s["q"], s["d"], s["start"], s["ua"], s["us"], s["acc"], s["tok"], s["ctx"], s["ctx"], dev_err=s["err"])
        between()
        mla.mla_release_pages(s["lens"], s["ctx"], None, s["table"], None, s["free"], s["mid"], num_pages, s["out"], s["left"], s["after"],
                              dev_err=s["err"])
        between()
        s["ctx"].copy_(s["left"])
        s["rng"].copy_(s["after"])
        between()

    a, b = state(), state()
    for s in (a, b):                                      # the prompts' pages: a plan of their tokens
        ctx = s["ctx"].clone()
        wide = e(int(ctx.sum()))
        mla.mla_plan_chunks(dev([0] * B), ctx, req, s["page_table"], s["free"], s["rng"], num_pages, s["table"], s["start"], s["lens"],
                            wide, wide.clone(), wide.clone(), s["head"], dev_err=s["err"])
        s["rng"][:1].copy_(s["head"])
    step(state(), torch.cuda.synchronize)                 # loads the kernels before the capture
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step(a, lambda: None)
    seen = set()
    for turn in range(15):
        logits = 2 * torch.randn((rows, V), generator=g)
        p, q = torch.softmax(logits, -1), torch.softmax(logits + 0.5 * torch.randn((rows, V), generator=g), -1)
        d, ua, us = torch.multinomial(q, 1, generator=g)[:, 0].int(), torch.rand(rows, generator=g), torch.rand(B, generator=g)
        for s in (a, b):
            for name, x in (("p", p), ("q", q), ("d", d), ("ua", ua), ("us", us)):
                s[name].copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        step(b, torch.cuda.synchronize)
        torch.cuda.synchronize()
        for name in ("acc", "tok", "ctx", "rng", "page_table", "free", "table", "out", "err"):
            assert torch.equal(a[name], b[name]), (turn, name)
        seen |= set(a["acc"].tolist())
        used = [int(x) for b_, m in enumerate(a["ctx"].tolist()) for x in a["out"][b_, : -(-m // 64)]]
        h, t = a["rng"].tolist()
        assert sorted(used + a["free"][h:t].tolist()) == list(range(num_pages))
    assert a["err"].item() == 0 and len(seen) >= 3
    assert np.all(a["ctx"].cpu().numpy() >= [55, 76, 141])
