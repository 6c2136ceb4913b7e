"""Plain 64-bit forms of the calls behind a step's attention (draft
verification, attention weight, selection, page release, moving tokens), and
the tolerance of the one that computes real numbers."""

import math

import numpy as np
import torch

PAGE = 64


def positive(x):
    return np.where((x > 0) & (x < math.inf), x, 0.0)


def verify(target, draft, drafts, start, u_acc, u_samp, width, lens=None):
    """target, draft (or None): float64 [rows, vocab] numpy arrays."""
    B, rows, V = len(start) - 1, target.shape[0], target.shape[1]
    acc, toks, kept, err = np.zeros(B, np.int32), np.full((B, width), -1, np.int32), None, 0
    kept = None if lens is None else np.array(lens, np.int32)
    if any(not 0 <= start[b] <= start[b + 1] <= rows for b in range(B)):
        return acc, toks, kept, 4
    for b in range(B):
        r0, n = start[b], start[b + 1] - start[b]
        if n == 0:
            continue
        if n > width:
            err |= 4
            continue
        passed = []
        for r in range(r0, r0 + n - 1):
            d = int(drafts[r])
            if not 0 <= d < V:
                err |= 32
                passed.append(False)
                continue
            p = float(positive(target[r, d]))
            q = 1.0 if draft is None else float(positive(draft[r, d]))
            passed.append(float(np.float32(u_acc[r])) * q < p)
        j = passed.index(False) if False in passed else n - 1
        row = positive(target[r0 + j])
        w = row
        if j < n - 1:
            d = int(drafts[r0 + j])
            if draft is None:
                w = row.copy()
                if 0 <= d < V:
                    w[d] = 0.0
            else:
                w = np.maximum(row - positive(draft[r0 + j]), 0.0)
            if not w.sum() > 0:
                w = row
        u = float(np.float32(u_samp[b]))
        u = min(u, 1.0) if u > 0 else 0.0
        cum = np.cumsum(w)
        some = np.nonzero(w)[0]
        pick = -1
        if some.size:
            over = np.nonzero((cum > u * cum[-1]) & (w > 0))[0]
            pick = int(over[0]) if over.size else int(some[-1])
        else:
            err |= 32
        acc[b] = j
        toks[b, :j] = drafts[r0:r0 + j]
        toks[b, j] = pick
        if kept is not None:
            kept[b] -= n - 1 - j
            if kept[b] < 0:
                err, kept[b] = err | 4, 0
    return acc, toks, kept, err


def select(mass, num_pages, table, lens, keep, sinks, recent, max_keep):
    """mass float32 [num_pages * 64] -> kept [B, max_keep], kept_lens, error bits."""
    B, P = table.shape
    kept, out, err = np.full((B, max_keep), -1, np.int32), np.zeros(B, np.int32), 0
    for b in range(B):
        L, K = int(lens[b]), int(keep[b])
        cut = True
        if not 0 <= L <= P * PAGE:
            err, L, cut = err | 4, 0, False
        elif K < 0 or (K < L and K > max_keep):
            err, cut = err | 4, False
        if not cut or K >= L:
            out[b] = L
            m = min(L, max_keep)
            kept[b, :m] = np.arange(m)
            continue
        out[b] = K
        s = min(sinks, K)
        r = min(recent, K - s)
        if K > 0:
            pages = table[b, : -(-L // PAGE)]
            bad = (pages < 0) | (pages >= num_pages)
            if bad.any():
                err |= 2
            at = np.where(bad, 0, pages).astype(np.int64)[:, None] * PAGE + np.arange(PAGE)
            m = mass[at].astype(np.float64)
            lowest = np.isnan(mass[at]) | bad[:, None]
            m[lowest] = -math.inf
            m, lowest = m.reshape(-1)[:L], lowest.reshape(-1)[:L]
            mid = np.arange(s, L - r)
            order = sorted(mid.tolist(), key=lambda t: (lowest[t], -m[t], t))[: K - s - r]
            kept[b, :K] = sorted(list(range(s)) + list(range(L - r, L)) + order)
    return kept, out, err


def release(old, new, req, table, page_table, free, head, tail, num_pages, move):
    """page_table (numpy) and free (list) are changed in place."""
    B, P = table.shape
    out, lens = np.full((B, P), -1, np.int32), np.zeros(B, np.int32)
    err, took, gave, avail, space = 0, 0, 0, tail - head, head
    if head < 0 or tail < head or tail > len(free):
        err, avail, space = 2, 0, 0
    plan, full = [], False
    for b in range(B):
        o, n = int(old[b]), int(new[b])
        ok = True
        if move and (not 0 <= req[b] < page_table.shape[0] or list(req).count(req[b]) > 1):
            err, ok = err | 2, False
        if not 0 <= o <= P * PAGE or not 0 <= n <= o:
            err, ok = err | 4, False
            o = o if 0 <= o <= P * PAGE else 0
        n = n if ok else o
        take = -(-n // PAGE) if move and n < o else 0
        back = -(-o // PAGE) - (0 if move else -(-n // PAGE)) if n < o else 0
        if take or back:
            full = full or took + take > avail or gave + back - took - take > space
            if full:
                err, n, take, back = err | 16, o, 0, 0
        plan.append((o, n, take, back, took, gave, bool(move and n < o)))
        took, gave = took + take, gave + back
    source = list(free)
    for b, (o, n, take, back, t0, g0, moved) in enumerate(plan):
        was, now = -(-o // PAGE), -(-n // PAGE)
        ids = []
        for p in range(was):
            i = int(table[b, p])
            if not 0 <= i < num_pages:
                err, i = err | 2, -1
            ids.append(i)
        for j in range(back):
            free[head + took - gave + g0 + j] = ids[(0 if moved else now) + j]
        for p in range(now):
            i = ids[p]
            if moved:
                i = source[head + t0 + p]
                if not 0 <= i < num_pages:
                    err, i = err | 2, -1
                page_table[req[b], p] = i
            out[b, p] = i
        lens[b] = n
    return out, lens, [head + took - gave, tail], err


def mass(c, k, q_lat, q_pe, lse, ctx, scale):
    """One sequence, doubles: c [T, 512], k [T, 64] dequantized, q_lat [n, H,
    512], q_pe [n, H, 64], lse [n, H] -> (the weight of every token, its bound).

    The bound.  A score's products enter with operands of 22 bits (2^-22 each,
    and 2^-22 for a product of two low parts left out) and are summed in fp32:
    576 rounded additions at most, each off by half a step of a partial sum no
    larger than the sum of the magnitudes.  A value below fp16's normal range
    is off by 2^-25 in either operand (queries with the scale and log2 e in
    them).  The exponent's argument takes three fp32 roundings of |s| + |lse|, the
    exponential itself 2^-21, the sum of n H weights one rounding each."""
    T, n, H = c.shape[0], q_lat.shape[0], q_lat.shape[1]
    x, y = torch.cat([c, k], -1), torch.cat([q_lat, q_pe], -1)
    s = torch.einsum("nhc,tc->nht", y, x) * scale
    seen = torch.ones((n, T), dtype=torch.bool).tril(ctx)[:, None, :] & torch.isfinite(lse)[..., None]
    lse = torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[..., None]
    w = torch.where(seen, torch.exp(s - lse), torch.zeros_like(s))
    mag = torch.einsum("nhc,tc->nht", y.abs(), x.abs()) * scale
    tiny = 2.0 ** -25 * (y.abs().sum(-1)[..., None] * scale * 1.45 + x.abs().sum(-1)) * 2
    ds = mag * (3 * 2.0 ** -22 + 576 * 2.0 ** -24) + tiny + 3 * 2.0 ** -24 * (s.abs() + lse.abs()) * 1.45
    off = (w * (torch.expm1(ds) + 2.0 ** -21)).sum((0, 1))
    total = w.sum((0, 1))
    return total, 1.01 * off + n * H * 2.0 ** -24 * total + 1e-37
