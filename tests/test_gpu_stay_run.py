"""The calls behind a step's attention together, as a program uses them: steps
of speculative decoding (plan, append, attention, verification, release) and a
cache kept within a budget (attention weight, selection, release, move),
against the same steps on the host."""

import math
import random

import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests import _stay_reference as R
from tests._helpers import F_INT4, F_INT4S, F_INT8

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module")
def mla():
    import mla_latent_kv_append_gb300 as m
    return m


def dev(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def e(*s):
    return torch.full(s, 77, dtype=torch.int32, device="cuda")


class Server:
    """The library's side: pools of two layers, page tables and a free list on
    the GPU.  The host's side: what every cached token of every request was."""

    def __init__(self, mla, B, P, num_pages, lf, kf, H=16, layers=2, seed=0):
        self.mla, self.B, self.P, self.H, self.num_pages, self.lf, self.kf = mla, B, P, H, num_pages, lf, kf
        self.g = torch.Generator().manual_seed(seed)
        self.caches = [mla.CacheLayer(num_pages, lf, kf) for _ in range(layers)]
        self.mass = [torch.zeros(num_pages * 64, device="cuda") for _ in range(layers)]
        self.req = dev(random.Random(seed).sample(range(B + 2), B))
        self.page_table = torch.full((B + 2, P), -1, dtype=torch.int32, device="cuda")
        self.free = dev(list(range(num_pages)))
        self.range = dev([0, num_pages])
        self.ctx = dev([0] * B)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.tokens = [[[] for _ in range(B)] for _ in range(layers)]      # (c, k) rows, host
        self.weight = [[[] for _ in range(B)] for _ in range(layers)]      # accumulated, host, doubles

    def rand(self, *s):
        return torch.randn(s, generator=self.g)

    def plan(self, new):
        """Block tables and slots of a step with these new tokens, appended to every layer."""
        n = sum(new)
        self.new = new
        self.table, self.start, self.lens, slot, head = e(self.B, self.P), e(self.B + 1), e(self.B), e(n), e(1)
        self.mla.mla_plan_chunks(self.ctx, dev(new), self.req, self.page_table, self.free, self.range, self.num_pages, self.table,
                                 self.start, self.lens, e(n), e(n), slot, head, dev_err=self.err)
        self.range = torch.stack([head[0], self.range[1]])
        for cache, tokens, weight in zip(self.caches, self.tokens, self.weight):
            c, k = self.rand(n, 512).bfloat16(), self.rand(n, 64).bfloat16()
            self.mla.mla_cache_append(cache, c.cuda(), k.cuda(), slot, dev_err=self.err)
            d = Q.quantize_token_rows(c.float().numpy(), k.float().numpy(), self.lf, self.kf)
            rows = np.concatenate([np.asarray(d["c_hat"], np.float64), np.asarray(d["kpe_hat"], np.float64)], 1)
            at = 0
            for b, m in enumerate(new):
                tokens[b] += list(rows[at:at + m])
                weight[b] += [0.0] * m
                at += m

    def release(self, new_lens, move):
        out, lens, rng = e(self.B, self.P), e(self.B), e(2)
        self.mla.mla_release_pages(self.lens, new_lens, self.req, self.table, self.page_table, self.free, self.range, self.num_pages, out,
                                   lens, rng, move=move, dev_err=self.err)
        self.range, self.ctx = rng, lens
        return out

    def check_pages(self, table):
        lens = self.ctx.tolist()
        t = table.cpu().numpy()
        used = [int(t[b, p]) for b in range(self.B) for p in range(-(-lens[b] // 64))]
        h, tail = self.range.tolist()
        assert sorted(used + self.free[h:tail].tolist()) == list(range(self.num_pages))

    def attend(self, layer, table):
        """The decode over the requests' caches gives the attention of the host's tokens."""
        mla, B, H = self.mla, self.B, self.H
        q_lat, q_pe = self.rand(B, H, 512) * 0.5, self.rand(B, H, 64).bfloat16()
        ws = torch.empty(mla.mla_decode_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
        o, lse = torch.empty((B, H, 512), device="cuda"), torch.empty((B, H), device="cuda")
        torch.cuda.synchronize()
        mla.mla_decode_absorbed(self.caches[layer], q_lat.cuda(), q_pe.cuda(), table, self.ctx, ws, o, lse, self.err)
        o = o.double().cpu()
        for b in range(B):
            if not self.tokens[layer][b]:
                continue
            x = torch.from_numpy(np.array(self.tokens[layer][b]))
            s = torch.cat([q_lat[b].double(), q_pe[b].double()], -1) @ x.t() * SCALE
            want = torch.softmax(s, -1) @ x[:, :512]
            # the decode's documented bound: 2e-3 of the row's largest value
            assert (o[b] - want).abs().amax() <= 2e-3 * want.abs().amax()


def test_speculative_steps(mla):
    B, V, P = 5, 300, 6
    s = Server(mla, B, P, 40, F_INT8, F_INT8, seed=1)
    r = random.Random(2)
    s.plan([r.randint(50, 130) for _ in range(B)])
    s.ctx = s.lens.clone()
    seen = set()
    for step in range(12):
        drafts = [r.randint(0, 4) for _ in range(B)]
        room = [P * 64 - int(c) for c in s.ctx.tolist()]
        drafts = [min(d, m - 1) for d, m in zip(drafts, room)]
        s.plan([d + 1 for d in drafts])
        rows = sum(drafts) + B
        logits = 2 * s.rand(rows, V)
        target, draft = torch.softmax(logits, -1), torch.softmax(logits + 0.5 * s.rand(rows, V), -1)
        tok = torch.multinomial(draft, 1, generator=s.g)[:, 0].int()
        ua, us = torch.rand(rows, generator=s.g), torch.rand(B, generator=s.g)
        acc, out, kept = e(B), e(B, 5), e(B)
        mla.mla_verify_drafts(target.cuda(), draft.cuda(), tok.cuda(), s.start, ua.cuda(), us.cuda(), acc, out, seq_lens=s.lens,
                              kept_lens=kept, dev_err=s.err)
        want = R.verify(target.double().numpy(), draft.double().numpy(), tok.numpy(), s.start.tolist(), ua.numpy(), us.numpy(), 5,
                        s.lens.tolist())
        table = s.release(kept, move=False)
        torch.cuda.synchronize()
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[1])
        assert s.ctx.tolist() == want[2].tolist() and s.err.item() == 0
        for tokens in s.tokens:
            for b in range(B):
                del tokens[b][s.ctx[b].item():]
        seen |= set(want[0].tolist())
        s.check_pages(table)
    s.attend(0, table)
    s.attend(1, table)
    assert len(seen) >= 3


@pytest.mark.parametrize("lf,kf", [(F_INT8, F_INT8), (F_INT4, F_INT4S)], ids=["int8", "int4"])
def test_a_cache_within_its_budget(mla, lf, kf):
    """Prompts, then decode steps that add up every token's attention weight;
    every few steps the requests over budget are cut to their heaviest tokens."""
    B, P, H, budget, sinks, recent = 4, 8, 16, 120, 4, 16
    s = Server(mla, B, P, 60, lf, kf, H=H, seed=3)
    r = random.Random(4)
    s.plan([r.randint(40, 300) for _ in range(B)])
    s.ctx = s.lens.clone()
    decay = 0.9
    table = s.table
    ws = torch.empty(mla.mla_mass_workspace_bytes(B, B, H, 1), dtype=torch.uint8, device="cuda")
    dws = torch.empty(mla.mla_decode_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
    counted = dev([0] * B)                                # the prompts' tokens have no weight yet
    cuts = 0
    for step in range(9):
        s.plan([1] * B)
        start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        for layer, cache in enumerate(s.caches):
            q_lat, q_pe = s.rand(B, H, 512) * 0.5, s.rand(B, H, 64).bfloat16()
            o, lse = torch.empty((B, H, 512), device="cuda"), torch.empty((B, H), device="cuda")
            torch.cuda.synchronize()                      # the decode reads the lengths during the launch overlap
            mla.mla_decode_absorbed(cache, q_lat.cuda(), q_pe.cuda(), s.table, s.lens, dws, o, lse, s.err)
            mla.mla_token_mass(cache, q_lat.cuda(), q_pe.cuda(), lse, s.table, start, s.lens, ws, s.mass[layer], max_new=1, decay=decay,
                               counted=counted if step == 0 else None, dev_err=s.err)
            lse = lse.double().cpu()
            for b in range(B):
                x = torch.from_numpy(np.array(s.tokens[layer][b]))
                w, _ = R.mass(x[:, :512], x[:, 512:], q_lat[b:b + 1].double(), q_pe[b:b + 1].double(), lse[b:b + 1], x.shape[0] - 1, SCALE)
                old = np.array(s.weight[layer][b]) * float(np.float32(decay))
                if step == 0:
                    old[:] = 0.0
                s.weight[layer][b] = list(old + w.numpy())
        s.ctx = s.lens
        if step % 3 != 2:
            continue
        cuts += 1
        lens = s.lens.tolist()
        keep = dev([budget] * B)
        kept, kept_lens = [e(B, budget) for _ in s.caches], e(B)
        for layer in range(2):
            mla.mla_select_tokens(s.mass[layer], s.table, s.lens, keep, kept[layer], kept_lens, sinks=sinks, recent=recent, dev_err=s.err)
        old_lens = s.lens
        new_table = s.release(kept_lens, move=True)
        for layer, cache in enumerate(s.caches):
            mla.mla_move_tokens(cache, s.table, old_lens, kept[layer], s.ctx, new_table, mass=s.mass[layer], dev_err=s.err)
        torch.cuda.synchronize()
        assert s.err.item() == 0 and s.ctx.tolist() == [min(budget, n) for n in lens]
        table = new_table
        s.check_pages(table)
        t = table.cpu().numpy()
        for layer in range(2):
            mass = s.mass[layer].cpu().numpy().astype(np.float64)
            for b in range(B):
                n = lens[b]
                if n > budget:
                    w = np.array(s.weight[layer][b])
                    mid = sorted(range(sinks, n - recent), key=lambda i: (-w[i], i))[: budget - sinks - recent]
                    want = sorted(list(range(sinks)) + mid + list(range(n - recent, n)))
                    got = kept[layer][b].tolist()
                    # the GPU's fp32 weights may order two that lie within 1e-4 of each other the other way
                    edge = w[mid[-1]]
                    assert all(abs(w[i] - edge) <= 1e-4 * edge for i in set(got) ^ set(want))
                    s.tokens[layer][b] = [s.tokens[layer][b][i] for i in got]
                    s.weight[layer][b] = [s.weight[layer][b][i] for i in got]
                j = np.arange(len(s.tokens[layer][b]))
                have = mass[t[b, j // 64].astype(np.int64) * 64 + j % 64]
                # three steps of sums near 1e-3 .. 1: each within 1e-5 of itself, and the smallest within 1e-6
                assert np.allclose(have, s.weight[layer][b], rtol=1e-4, atol=1e-6)
            s.attend(layer, table)
    assert cuts == 3


def test_a_cut_in_a_graph(mla):
    """Selection, release and move captured once and replayed with other
    lengths, against the calls one by one on a copy."""
    B, P, num_pages, budget = 3, 6, 50, 90
    s = Server(mla, B, P, num_pages, F_INT8, F_INT8, layers=1, seed=5)
    s.plan([300, 140, 128])                               # pages for every replay below
    cache, keep = s.caches[0], dev([budget] * B)
    kept, kept_lens, out, lens, rng = e(B, budget), e(B), e(B, P), e(B), e(2)
    state = [cache.pool, s.mass[0], s.table, s.lens, s.page_table, s.free, s.range]

    def cut():
        mla.mla_select_tokens(s.mass[0], s.table, s.lens, keep, kept, kept_lens, sinks=2, recent=8, dev_err=s.err)
        mla.mla_release_pages(s.lens, kept_lens, s.req, s.table, s.page_table, s.free, s.range, num_pages, out, lens, rng, move=True,
                              dev_err=s.err)
        mla.mla_move_tokens(cache, s.table, s.lens, kept, lens, out, mass=s.mass[0], dev_err=s.err)

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    first = [t.clone() for t in state]
    cut()                                                 # loads the kernels before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        cut()
    for lengths in ([300, 140, 64], [91, 90, 0], [200, 1, 128]):
        results = []
        for call in (g.replay, cut):
            for t, v in zip(state, first):
                t.copy_(v)
            s.mass[0].copy_(torch.rand(num_pages * 64, generator=torch.Generator().manual_seed(6)))
            s.lens.copy_(dev(lengths))
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
            results.append([t.clone() for t in state + [kept, kept_lens, out, lens, rng]])
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert results[0][-2].tolist() == [min(budget, n) for n in lengths]
    assert s.err.item() == 0
