"""Plain 64-bit forms of the serving-step operators (plan, rotary positions,
chunk attention), and the tolerances that follow from their roundings."""

import math

import numpy as np
import torch

PAGE = 64
SCALE = 1.0 / math.sqrt(192.0)
U16 = 2.0 ** -11           # largest relative error of one rounding to fp16
UB = 2.0 ** -8             # and to bf16


def plan(ctx, new, req, table, free, head, tail, num_pages, n):
    """Python twin of the step plan: lists and int lists of lists in, a dict
    of numpy int32 arrays out; table is changed in place."""
    B, P = len(ctx), table.shape[1]
    out = {"block_table": np.full((B, P), -1, np.int32), "q_start": np.zeros(B + 1, np.int32),
           "seq_lens": np.zeros(B, np.int32), "positions": np.zeros(n, np.int32),
           "token_req": np.full(n, -1, np.int32), "slot": np.full(n, -1, np.int32)}
    err, start, first, taken = 0, 0, 0, 0
    avail = tail - head
    if head < 0 or tail > len(free) or avail < 0:
        err, avail = err | 2, 0
    for b in range(B):
        c, m, r = int(ctx[b]), int(new[b]), int(req[b])
        ok = True
        if not 0 <= r < table.shape[0] or list(req).count(r) > 1:
            err, ok = err | 2, False
        if c < 0 or m < 0 or c + m > P * PAGE:
            err, ok = err | 4, False
            m = max(m, 0)
        out["q_start"][b] = min(start, n)
        rows = range(min(start, n), min(start + m, n))
        start += m
        if start > n:
            err, ok = err | 4, False
        if ok:
            old, now = -(-c // PAGE), -(-(c + m) // PAGE)
            if now > old and first + now - old > avail:
                err, ok = err | 16, False
            else:
                for p in range(old, now):
                    i = free[head + first + p - old]
                    table[r, p] = i if 0 <= i < num_pages else -1
                if now > old:
                    taken = max(taken, first + now - old)
            first += now - old
        for i in rows:
            out["token_req"][i] = b
        if ok:
            out["seq_lens"][b] = c + m
            for p in range(now):
                i = table[r, p]
                if not 0 <= i < num_pages:
                    err |= 2
                    i = -1
                out["block_table"][b, p] = i
            for k, i in enumerate(rows):
                pos = c + k
                out["positions"][i] = pos
                pg = out["block_table"][b, pos // PAGE]
                out["slot"][i] = pg * PAGE + pos % PAGE if pg >= 0 else -1
    out["q_start"][B] = min(start, n)
    out["free_head"] = np.array([head + taken], np.int32)
    return out, err


def rope(x, pos, inv_freq, axis, interleaved, inverse, amp):
    """x [n, ..., 64] double, pos [axes, n] ints, inv_freq [32] -> double."""
    ang = pos.double()[list(axis)].t() * inv_freq.double()[None, :]
    if inverse:
        ang = -ang
    shape = (ang.shape[0],) + (1,) * (x.dim() - 2) + (32,)
    c, s = (amp * ang.cos()).reshape(shape), (amp * ang.sin()).reshape(shape)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).reshape(x.shape)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def rope_bound(y, x, amp):
    """Largest error of a rotated value: two fp32 products of fp32 sines (an
    angle off by 2e-6, the sines' and amplitude's rounding: 3e-6 in all),
    summed, rounded once to bf16 (a value whose terms cancel has the terms'
    error, hence the row's largest entry)."""
    mag = abs(amp) * x.abs().amax(-1, keepdim=True) * 2
    return UB * y.abs() + 4e-6 * mag + 1e-30


def chunk(c, k, q_nope, q_pe, w_uk, w_uv, ctx, scale=SCALE, skip=None):
    """One sequence, doubles: c [T, 512], k [T, 64] dequantized; q [n, H, ..];
    -> (o [n, H, 128], elementwise bound, squared 2-norm of the expected
    error).  skip: bool [T], tokens that contribute nothing.

    The bound.  Each of the operands of the two products (absorbed: q_lat and
    c against c; expanded: the per-head key and value, made from a rounded c)
    is rounded once to fp16, P too, and o once to bf16; fp32 sums add 2^-20.
    A score is then off by at most ds = u (2 sum |q_lat c| + sum |q_nope K| +
    2 sum |q_pe k|) scale, its weight by a factor e^(+-2 ds) after
    normalisation, and the output by
      (e^(2 ds) - 1 + 2 u) sum w |v| + u sum w (|c| |W_UV|) + 2^-8 |o|.
    The expected error takes the same roundings as independent, uniform
    within their half steps (variance u^2 / 3 each)."""
    T, n, H = c.shape[0], q_nope.shape[0], q_nope.shape[1]
    out = torch.empty((n, H, 128), dtype=torch.float64)
    bound = torch.empty_like(out)
    mean2 = 0.0
    seen = torch.ones((n, T), dtype=torch.bool).tril(ctx)
    if skip is not None:
        seen &= ~skip[None, :]
    for h in range(H):
        ql = q_nope[:, h] @ w_uk[h]
        K, V = c @ w_uk[h].t(), c @ w_uv[h]
        s = (q_nope[:, h] @ K.t() + q_pe[:, h] @ k.t()) * scale
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        w = torch.where(l > 0, p / l, torch.zeros_like(p))
        o = w @ V
        sabs = scale * (2 * ql.abs() @ c.abs().t() + q_nope[:, h].abs() @ K.abs().t() + 2 * q_pe[:, h].abs() @ k.abs().t())
        ds = U16 * 1.02 * (sabs * seen).amax(-1, keepdim=True)
        vabs, cw = w @ V.abs(), w @ (c.abs() @ w_uv[h].abs())
        out[:, h] = o
        bound[:, h] = (torch.expm1(2 * ds) + 2.1 * U16) * vabs + 1.1 * U16 * cw + 1.01 * UB * o.abs() + 1e-30
        s2 = scale ** 2 * (2 * (ql ** 2) @ (c ** 2).t() + (q_nope[:, h] ** 2) @ (K ** 2).t() + 2 * (q_pe[:, h] ** 2) @ (k ** 2).t())
        var = U16 ** 2 / 3 * ((w ** 2 * (s2 + 2)) @ (V ** 2) + (w ** 2) @ ((c ** 2) @ (w_uv[h] ** 2)))
        mean2 += float((var + UB ** 2 / 3 * o ** 2).sum())
    return out, bound, mean2
