"""What happens to the paged latent cache after a step's attention, as
operators with their plain forms: which of the cached tokens stay.

* verify:  drafted tokens against the target's probabilities (speculative
  sampling) from given random numbers, and the token sampled behind them;
* mass:    the attention weight that every cached token received from a
  step's queries, added to the weight it had;
* select:  the tokens of each sequence that stay in a smaller cache: the first
  ones, the latest ones and those with the most weight;
* pages:   page tables and the free list after requests got shorter, by
  dropping their last tokens or by moving the kept ones into fresh pages;
* move:    the kept tokens' cached values and weights into those pages.

A case is a dict of plain values; sequence lengths follow from its own
``lens_seed``, every tensor's values from the seed that prepare() gets.
"""

import math
import random

import numpy as np
import torch

own = False

D_C, D_R, PAGE, BLOCK = 512, 64, 64, 32
SCALE = 1.0 / math.sqrt(128 + D_R)

# (latent format, k_pe format) of a cache -> the library's format numbers
FORMATS = {"bf16": (0, 0), "int8": (1, 1), "int4": (2, 1), "int4_int4": (2, 3)}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one chat request with four drafted tokens, a small vocabulary: latency
        {"name": "verify_one", "op": "verify", "batch": 1, "drafts": 4, "vocab": 32003, "dtype": "fp32", "lookup": False, "lens_seed": 1},
        # a busy server: 256 requests with up to four drafts each, a large vocabulary
        {"name": "verify_busy", "op": "verify", "batch": 256, "drafts": 4, "vocab": 131072, "dtype": "fp32", "lookup": False, "lens_seed": 2},
        # one request's decode token
        {"name": "mass_decode_one", "op": "mass", "fmt": "int8", "heads": 16, "batch": 1, "ctx_lo": 4096, "ctx_hi": 4096, "new": 1,
         "fresh": False, "lens_seed": 3},
        # a decode batch of long contexts in the smallest format
        {"name": "mass_decode_long", "op": "mass", "fmt": "int4_int4", "heads": 16, "batch": 32, "ctx_lo": 32767, "ctx_hi": 32767, "new": 1,
         "fresh": False, "lens_seed": 4},
        # drafts being verified, ragged, at 64 heads
        {"name": "mass_drafts", "op": "mass", "fmt": "bf16", "heads": 64, "batch": 24, "ctx_lo": 1000, "ctx_hi": 16000, "new": 5,
         "fresh": False, "lens_seed": 5},
        # the last 32 queries of long prompts judge all their tokens, once
        {"name": "mass_window", "op": "mass", "fmt": "int8", "heads": 16, "batch": 4, "ctx_lo": 15000, "ctx_hi": 15968, "new": 32,
         "fresh": True, "lens_seed": 6},
        # one long request cut to a sixteenth
        {"name": "select_one", "op": "select", "batch": 1, "ctx_lo": 32768, "ctx_hi": 32768, "keep": 0.0625, "sinks": 4, "recent": 256,
         "lens_seed": 7},
        # a batch of them, ragged, cut to a quarter
        {"name": "select_batch", "op": "select", "batch": 64, "ctx_lo": 2000, "ctx_hi": 65536, "keep": 0.25, "sinks": 4, "recent": 512,
         "lens_seed": 8},
        # a few requests give back the pages of rejected drafts
        {"name": "pages_trim", "op": "pages", "batch": 32, "rows": 64, "max_pages": 512, "ctx_hi": 32000, "move": False, "lens_seed": 9},
        # an offline batch at the library's batch limit moves into a quarter of its pages
        {"name": "pages_move", "op": "pages", "batch": 4096, "rows": 5000, "max_pages": 640, "ctx_hi": 40000, "move": True, "lens_seed": 10},
        # one request's kept tokens, a sixteenth of them
        {"name": "move_one", "op": "move", "fmt": "int8", "batch": 1, "ctx_lo": 32768, "ctx_hi": 32768, "keep": 0.0625, "lens_seed": 11},
        # a batch that keeps a quarter, in the smallest format
        {"name": "move_batch", "op": "move", "fmt": "int4_int4", "batch": 32, "ctx_lo": 4000, "ctx_hi": 32768, "keep": 0.25, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["verify", "mass", "mass", "select", "pages", "move"])
    seed = rng.randint(0, 1 << 30)
    for _ in range(1000):
        if op == "verify":
            case = {"op": op, "batch": _log_int(rng, 1, 256), "drafts": rng.randint(0, 8), "vocab": _log_int(rng, 1000, 131072),
                    "dtype": rng.choice(sorted(TYPES)), "lookup": rng.random() < 0.25, "lens_seed": seed}
            if case["batch"] * (case["drafts"] + 1) * case["vocab"] <= 120_000_000:
                return case
            continue
        if op == "pages":
            return {"op": op, "batch": (b := _log_int(rng, 1, 4096)), "rows": b + rng.randint(0, 1000), "max_pages": _log_int(rng, 16, 640),
                    "ctx_hi": _log_int(rng, 64, 40000), "move": rng.random() < 0.5, "lens_seed": seed}
        hi = _log_int(rng, 16, 131072 if op == "select" else 65536)
        case = {"op": op, "batch": _log_int(rng, 1, 256), "ctx_lo": rng.randint(hi // 4, hi), "ctx_hi": hi, "lens_seed": seed}
        tokens = case["batch"] * hi
        if op == "select":
            case |= {"keep": round(rng.uniform(0.02, 1.0), 3), "sinks": rng.choice([0, 4, 64]), "recent": _log_int(rng, 1, 1024)}
            if tokens <= 4_000_000:
                return case
            continue
        case["fmt"] = rng.choice(sorted(FORMATS))
        if op == "move":
            case["keep"] = round(rng.uniform(0.02, 1.0), 3)
            if tokens <= 600_000:
                return case
            continue
        kind = rng.choice(["decode", "drafts", "window"])
        case |= {"heads": rng.choice([16, 32, 48, 64, 128]), "fresh": rng.random() < 0.3,
                 "new": {"decode": 1, "drafts": rng.randint(2, 9), "window": rng.randint(10, 64)}[kind]}
        w = work(case)
        if tokens <= 1_000_000 and w["bytes"] <= 6.1e8 and w["flops"] <= 3.6e10:
            return case
    raise RuntimeError("no case within the limits")


def _lens(case):
    r = random.Random(case["lens_seed"])
    lo, hi = case.get("ctx_lo", 1), case["ctx_hi"]
    return [hi if lo >= hi else int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) for _ in range(case["batch"])], r


def _mass_lens(case):
    """(cached tokens before the step, new tokens) of every sequence; the first has the most new ones."""
    ctx, r = _lens(case)
    new = [case["new"] if b == 0 or case["new"] > 9 else r.randint(1, case["new"]) for b in range(case["batch"])]
    return ctx, new


def _draft_lens(case):
    r = random.Random(case["lens_seed"])
    return [case["drafts"] if b == 0 else r.randint(case["drafts"] // 2, case["drafts"]) for b in range(case["batch"])]


def _keep_lens(case):
    lens, r = _lens(case)
    return lens, [max(1, min(n, int(n * case["keep"]))) for n in lens]


def _page_lens(case):
    r = random.Random(case["lens_seed"])
    cap = case["max_pages"] * PAGE
    old = [min(cap, int(math.exp(r.uniform(0, math.log(case["ctx_hi"] + 1))))) for _ in range(case["batch"])]
    if case["move"]:
        return old, [n if r.random() < 0.1 else max(1, n // 4) for n in old]
    return old, [max(0, n - r.choice([0, 0, 1, 2, 3, 5, 70])) for n in old]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


# ---------------------------------------------------------------------------
# the cache's bytes: pages of two 32-token blocks, fields and chunk order as
# the library's header documents them
# ---------------------------------------------------------------------------

def _layout(fmt):
    lf, kf = FORMATS[fmt]
    off, at = 0, {}
    at["row"] = {0: 2 * D_C, 1: D_C, 2: D_C // 2}[lf]
    off += BLOCK * at["row"]
    if lf:
        at["scale"], off = off, off + 32 * BLOCK * 4
    if lf == 2:
        at["zero"], off = off, off + 32 * BLOCK * 4
    at["krow"] = {0: 2 * D_R, 1: D_R, 3: D_R // 2}[kf]
    at["kpe"], off = off, off + BLOCK * at["krow"]
    if kf:
        at["kscale"], off = off, off + 8 * BLOCK * 4
    if lf:
        at["bound"], off = off, off + BLOCK * 4
    at["bytes"] = off
    return at


def _chunk_pos(row, kf=None, device="cuda"):
    """[32, chunks]: the stored position of 16-byte chunk c of block token u."""
    c = torch.arange(row // 16, device=device)[None, :]
    u = torch.arange(BLOCK, device=device)[:, None]
    if kf is None or kf == 0:
        return (c & ~7) | ((c ^ u) & 7)
    return c ^ ((u >> 1) & 3) if kf == 1 else c ^ ((u >> 2) & 1)


def _nibble_channels(device="cuda"):
    """[32]: the channel (of a chunk's 32) of nibble k of word j, at 8 j + k."""
    j = torch.arange(4, device=device)[:, None]
    k = torch.arange(8, device=device)[None, :]
    return (((k >> 1) & 1) * 16 + 4 * j + (k & 1) * 2 + (k >> 2)).reshape(-1)


def _unpack_nibbles(chunks):
    """uint8 [..., chunks, 16] -> nibble values [..., chunks * 32] in channel order."""
    w = chunks.reshape(*chunks.shape[:-1], 4, 4)
    n = torch.stack([w & 15, w >> 4], dim=-1).reshape(*chunks.shape[:-1], 32)
    out = torch.empty_like(n)
    out[..., _nibble_channels(chunks.device)] = n
    return out.reshape(*chunks.shape[:-2], -1)


def _pack_nibbles(v):
    """uint8 [..., channels] -> uint8 [..., channels / 32, 16]."""
    n = v.reshape(*v.shape[:-1], -1, 32)[..., _nibble_channels(v.device)].reshape(*v.shape[:-1], -1, 16, 2)
    return n[..., 0] | (n[..., 1] << 4)


def _sym(x, group, levels):
    g = x.reshape(*x.shape[:-1], -1, group)
    s = g.abs().amax(-1) / levels
    q = torch.where(s[..., None] > 0, torch.round(g / s[..., None]), torch.zeros_like(g)).clamp(-levels, levels)
    return q.reshape(x.shape), s


def _asym4(x):
    g = x.reshape(*x.shape[:-1], -1, 16)
    mn, mx = g.amin(-1), g.amax(-1)
    s = (mx - mn) / 15
    s = torch.where(s == 0, mn.abs(), s)
    z = torch.where(s > 0, torch.round(-mn / s), torch.zeros_like(s))
    q = torch.where(s[..., None] > 0, (torch.round(g / s[..., None]) + z[..., None]).clamp(0, 15), torch.zeros_like(g))
    return q.reshape(x.shape), s, z


def _put(blocks, off, value):
    """value [nb, ...] of any type into the blocks' bytes at off."""
    v = value.contiguous().view(torch.uint8).reshape(blocks.shape[0], -1)
    blocks[:, off:off + v.shape[1]] = v


def _fill(blocks, fmt, c, k):
    """Quantizes tokens c [nb, 32, 512], k [nb, 32, 64] (bf16) into blocks [nb, bytes]."""
    lf, kf = FORMATS[fmt]
    at = _layout(fmt)
    nb = blocks.shape[0]

    def chunked(raw, row, pos):
        raw = raw.reshape(nb, BLOCK, row // 16, 16)
        out = torch.empty_like(raw)
        out.scatter_(2, pos[None, :, :, None].expand_as(raw), raw)
        return out

    x = c.float()
    if lf == 0:
        raw = c.contiguous().view(torch.uint8)
    elif lf == 1:
        q, s = _sym(x, 16, 127)
        raw, bound = q.to(torch.int8).view(torch.uint8), s.amax(-1) * 127
        _put(blocks, at["scale"], s.transpose(1, 2))
    else:
        q, s, z = _asym4(x)
        raw, bound = _pack_nibbles(q.to(torch.uint8)), (s * ((z - 7.5).abs() + 7.5)).amax(-1)
        _put(blocks, at["scale"], s.transpose(1, 2))
        _put(blocks, at["zero"], z.transpose(1, 2))
    _put(blocks, 0, chunked(raw, at["row"], _chunk_pos(at["row"], device=c.device)))
    if lf:
        _put(blocks, at["bound"], bound)
    if kf == 0:
        raw = k.contiguous().view(torch.uint8)
    else:
        q, s = _sym(k.float(), 8, 127 if kf == 1 else 7)
        raw = q.to(torch.int8).view(torch.uint8) if kf == 1 else _pack_nibbles((q + 8).to(torch.uint8))
        _put(blocks, at["kscale"], s.transpose(1, 2))
    _put(blocks, at["kpe"], chunked(raw, at["krow"], _chunk_pos(at["krow"], kf, c.device)))


def _read(pool, fmt, pages, dtype):
    """Dequantized (c_hat [..., 512], kpe_hat [..., 64]) of the tokens of pages [...]; `dtype` float32 or float64."""
    lf, kf = FORMATS[fmt]
    at = _layout(fmt)
    blocks = pool.view(-1, 2 * at["bytes"])[pages.long()].reshape(-1, at["bytes"])
    nb = blocks.shape[0]

    def codes(off, row, pos):
        raw = blocks[:, off:off + BLOCK * row].reshape(nb, BLOCK, row // 16, 16)
        return raw.gather(2, pos[None, :, :, None].expand_as(raw))

    def field(off, groups):
        return blocks[:, off:off + groups * BLOCK * 4].contiguous().view(torch.float32).reshape(nb, groups, BLOCK).transpose(1, 2)

    raw = codes(0, at["row"], _chunk_pos(at["row"], device=pool.device))
    if lf == 0:
        c = raw.reshape(nb, BLOCK, -1).view(torch.bfloat16).to(dtype)
    elif lf == 1:
        q = raw.reshape(nb, BLOCK, 32, 16).view(torch.int8).to(dtype)
        c = (q * field(at["scale"], 32).to(dtype)[..., None]).reshape(nb, BLOCK, D_C)
    else:
        q = _unpack_nibbles(raw).to(dtype).reshape(nb, BLOCK, 32, 16)
        c = ((q - field(at["zero"], 32).to(dtype)[..., None]) * field(at["scale"], 32).to(dtype)[..., None]).reshape(nb, BLOCK, D_C)
    raw = codes(at["kpe"], at["krow"], _chunk_pos(at["krow"], kf, pool.device))
    if kf == 0:
        k = raw.reshape(nb, BLOCK, -1).view(torch.bfloat16).to(dtype)
    else:
        q = raw.reshape(nb, BLOCK, D_R).view(torch.int8).to(dtype) if kf == 1 else _unpack_nibbles(raw).to(dtype) - 8
        k = (q.reshape(nb, BLOCK, 8, 8) * field(at["kscale"], 8).to(dtype)[..., None]).reshape(nb, BLOCK, D_R)
    lead = pages.shape[:-1]
    return c.reshape(*lead, -1, D_C), k.reshape(*lead, -1, D_R)


def _pool(fmt, num_pages, g):
    """A pool of latents as they come from behind a norm: unit-sized channels of
    uneven gain, some far from zero, a few large ones."""
    at = _layout(fmt)
    gain = torch.exp(0.6 * torch.randn(D_C, generator=g, device="cuda"))
    mean = 0.5 * torch.randn(D_C, generator=g, device="cuda")
    gain[torch.randperm(D_C, generator=g, device="cuda")[:4]] *= 6
    pool = torch.zeros((num_pages, 2 * at["bytes"]), dtype=torch.uint8, device="cuda")
    step = 4096
    for p in range(0, num_pages, step):
        part = pool[p:p + step].view(-1, at["bytes"])
        c = (mean + gain * torch.randn((part.shape[0], BLOCK, D_C), generator=g, device="cuda")).bfloat16()
        k = torch.randn((part.shape[0], BLOCK, D_R), generator=g, device="cuda").bfloat16()
        _fill(part, fmt, c, k)
    return pool.view(-1)


# ---------------------------------------------------------------------------
# prepare
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return {"verify": _prepare_verify, "mass": _prepare_mass, "select": _prepare_select, "pages": _prepare_pages,
            "move": _prepare_move}[case["op"]](case, g)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _ints([sum(lens[:b]) for b in range(len(lens) + 1)]) if len(lens) < 512 else \
        torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(_ints(lens), 0).int()])


def _table(lens, max_pages, first_id, g, spare=0):
    """int32 [B, max_pages] of page ids in random order, -1 behind each sequence's last; the spare ids."""
    pages = [_pages(t) for t in lens]
    perm = torch.randperm(sum(pages) + spare, generator=g, device="cuda").int() + first_id
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(max_pages, device="cuda")[None, :] < _ints(pages)[:, None]
    table[used] = perm[: sum(pages)]
    return table, perm[sum(pages):].contiguous()


def _prepare_verify(case, g):
    """Target rows as a model's at temperature 1 over a Zipf-like vocabulary,
    drafts drawn from a smaller model's distribution near the target's."""
    drafts = _draft_lens(case)
    n, v, dt = sum(drafts) + case["batch"], case["vocab"], TYPES[case["dtype"]]
    prior = -1.1 * torch.log1p(torch.randperm(v, generator=g, device="cuda").float())
    target = torch.empty((n, v), dtype=dt, device="cuda")
    draft = None if case["lookup"] else torch.empty((n, v), dtype=dt, device="cuda")
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    step = max(1, 100_000_000 // v)
    for r in range(0, n, step):
        m = min(step, n - r)
        logits = prior + 1.5 * torch.randn((m, v), generator=g, device="cuda")
        target[r:r + m] = torch.softmax(logits, -1).to(dt)
        q = torch.softmax(logits + 0.7 * torch.randn((m, v), generator=g, device="cuda"), -1).to(dt)
        u = torch.rand(m, generator=g, device="cuda").double()
        cum = torch.cumsum(q.double(), -1)
        tokens[r:r + m] = torch.searchsorted(cum, (u * cum[:, -1])[:, None], right=True)[:, 0].clamp(max=v - 1).int()
        if draft is not None:
            draft[r:r + m] = q
    return {"case": case, "target": target, "draft": draft, "tokens": tokens, "row_start": _starts([d + 1 for d in drafts]),
            "u_accept": torch.rand(n, generator=g, device="cuda"), "u_sample": torch.rand(case["batch"], generator=g, device="cuda"),
            "seq_lens": _ints([1000 + d + 1 for d in drafts])}


def _prepare_mass(case, g):
    ctx, new = _mass_lens(case)
    n, h, lens = sum(new), case["heads"], [c + m for c, m in zip(ctx, new)]
    max_pages = max(_pages(t) for t in lens)
    table, _ = _table(lens, max_pages, 0, g)
    num_pages = sum(_pages(t) for t in lens)
    pool = _pool(case["fmt"], num_pages, g)
    s = {"case": case, "pool": pool, "num_pages": num_pages, "table": table, "max_new": max(new), "ctx": _ints(ctx), "n": n,
         "q_start": _starts(new), "seq_lens": _ints(lens),
         # absorbed queries of unit-sized ones and weights of 1 / sqrt(512)
         "q_lat": torch.randn((n, h, D_C), generator=g, device="cuda") * math.sqrt(128 / D_C),
         "q_pe": torch.randn((n, h, D_R), generator=g, device="cuda").bfloat16(),
         # some steps' worth of weight, heavier on a few tokens
         "mass": torch.rand(num_pages * PAGE, generator=g, device="cuda").pow_(-0.5).sub_(1).mul_(8.0 * h * case["batch"] / sum(lens)),
         "counted": _ints([0] * case["batch"]) if case["fresh"] else None, "decay": 1.0 if case["fresh"] else 0.98}
    sc, _ = _scores(s, torch.float32)
    rows = torch.logsumexp(sc, -1)                                   # [B, new, H]: what the attention returned
    s["lse"] = rows[_real_rows(s)].contiguous()
    return s


def _prepare_select(case, g):
    lens, keep = _keep_lens(case)
    max_pages = max(_pages(t) for t in lens)
    table, _ = _table(lens, max_pages, 0, g)
    mass = torch.rand(sum(_pages(t) for t in lens) * PAGE, generator=g, device="cuda").pow_(-0.7).sub_(1)
    # tokens of equal weight are common: many were never looked at
    mass = torch.where(mass < 0.3, torch.zeros_like(mass), mass)
    return {"case": case, "mass": mass, "table": table, "seq_lens": _ints(lens), "keep": _ints(keep), "max_keep": max(keep)}


def _prepare_pages(case, g):
    old, new = _page_lens(case)
    need = sum(_pages(n) for n, o in zip(new, old) if n < o) if case["move"] else 0
    table, spare = _table(old, case["max_pages"], 0, g, spare=need + 1000)
    used = sum(_pages(t) for t in old)
    rows = torch.randperm(case["rows"], generator=g, device="cuda")[: case["batch"]].int()
    page_table = torch.full((case["rows"], case["max_pages"]), -1, dtype=torch.int32, device="cuda")
    page_table[rows.long()] = table
    # the list's front was given out, its places hold old ids
    head = used + 5
    free = torch.cat([torch.arange(head, dtype=torch.int32, device="cuda"), spare]).contiguous()
    return {"case": case, "old": _ints(old), "new": _ints(new), "req": rows, "table": table, "page_table": page_table, "free": free,
            "free_range": _ints([head, free.numel()]), "num_pages": used + spare.numel()}


def _prepare_move(case, g):
    lens, keep = _keep_lens(case)
    max_pages = max(_pages(t) for t in lens)
    moved = [k if k < t else 0 for k, t in zip(keep, lens)]
    table, spare = _table(lens, max_pages, 0, g, spare=sum(_pages(k) for k in moved))
    num_pages = sum(_pages(t) for t in lens) + spare.numel()
    pool = _pool(case["fmt"], num_pages, g)
    max_keep = max(keep)
    # the kept ones: uniform among a sequence's tokens, increasing
    width = max(lens)
    order = torch.rand((case["batch"], width), generator=g, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    order = torch.where(col < _ints(lens)[:, None], order, torch.full_like(order, 2.0))
    pick = torch.argsort(order, -1)[:, :max_keep]
    pick = torch.where(col[:, :max_keep] < _ints(keep)[:, None], pick, torch.full_like(pick, 1 << 40)).sort(-1).values
    kept = torch.where(pick < (1 << 40), pick, torch.full_like(pick, -1)).int().contiguous()
    dst = torch.full_like(table, -1)
    dst[torch.arange(max_pages, device="cuda")[None, :] < _ints([_pages(k) for k in moved])[:, None]] = spare
    stays = _ints([int(k == t) for k, t in zip(keep, lens)])[:, None] > 0
    return {"case": case, "pool": pool, "num_pages": num_pages, "table": table, "dst": torch.where(stays, table, dst).contiguous(),
            "seq_lens": _ints(lens), "kept": kept, "lens": _ints(keep),
            "mass": torch.rand(num_pages * PAGE, generator=g, device="cuda")}


# ---------------------------------------------------------------------------
# run
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"verify": _own_verify, "mass": _own_mass, "select": _own_select, "pages": _own_pages, "move": _own_move}[op](state)
    return {"verify": _plain_verify, "mass": _plain_mass, "select": _plain_select, "pages": _plain_pages, "move": _plain_move}[op](state)


def _positive(x):
    return torch.where((x > 0) & (x < math.inf), x, torch.zeros_like(x))


def _plain_verify(s):
    """Sums and comparisons in 64 bits: a rounded one would pick a neighbour."""
    case, start = s["case"], s["row_start"].long()
    batch, width = case["batch"], case["drafts"] + 1
    i = torch.arange(width, device="cuda")[None, :]
    n = (start[1:] - start[:-1])[:, None]
    row = (start[:-1, None] + i).clamp(max=s["target"].shape[0] - 1)
    d = s["tokens"].long()[row]
    p = _positive(s["target"][row, d].double())
    q = torch.ones_like(p) if s["draft"] is None else _positive(s["draft"][row, d].double())
    passed = (s["u_accept"].double()[row] * q < p) & (i < n - 1)
    accepted = torch.cumprod(passed.long(), 1).sum(1)
    at = torch.gather(row, 1, accepted[:, None])[:, 0]
    rejected = (accepted < n[:, 0] - 1)[:, None]
    full = _positive(s["target"][at].double())
    if s["draft"] is None:
        rest = full.clone().scatter_(1, torch.gather(d, 1, accepted[:, None]), 0.0)
    else:
        rest = (full - _positive(s["draft"][at].double())).clamp_(min=0)
    rest = torch.where(rejected & (rest.sum(1, keepdim=True) > 0), rest, full)
    cum = torch.cumsum(rest, 1)
    u = s["u_sample"].double().clamp(0, 1)
    last = (torch.arange(case["vocab"], device="cuda") * (rest > 0)).amax(1)
    pick = torch.minimum(torch.searchsorted(cum, (u * cum[:, -1])[:, None], right=True)[:, 0], last)
    tokens = torch.where(i < accepted[:, None], d, torch.where(i == accepted[:, None], pick[:, None], torch.full_like(d, -1)))
    return {"accepted": accepted.int(), "tokens": tokens.int(), "kept_lens": (s["seq_lens"] - (n[:, 0] - 1 - accepted)).int()}


def _own_verify(s):
    import mla_latent_kv_append_gb300 as mla
    if "out" not in s:
        b = s["case"]["batch"]
        e = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out"] = {"accepted": e(b), "tokens": e(b, s["case"]["drafts"] + 1), "kept_lens": e(b)}
    o = s["out"]
    mla.mla_verify_drafts(s["target"], s["draft"], s["tokens"], s["row_start"], s["u_accept"], s["u_sample"], o["accepted"],
                          o["tokens"], seq_lens=s["seq_lens"], kept_lens=o["kept_lens"])
    return o


def _real_rows(s):
    i = torch.arange(s["max_new"], device="cuda")[None, :]
    return i < (s["q_start"][1:] - s["q_start"][:-1]).long()[:, None]


def _scores(s, dtype):
    """[B, new, H, T]: scaled scores, -inf where a query does not see the key; and whether token t is the sequence's."""
    n = s["q_start"][1:].long() - s["q_start"][:-1].long()
    i = torch.arange(s["max_new"], device="cuda")
    row = (s["q_start"][:-1, None].long() + i[None, :]).clamp(max=s["n"] - 1)
    c, k = _read(s["pool"], s["case"]["fmt"], s["table"].clamp(min=0), dtype)
    y = torch.cat([s["q_lat"].to(dtype)[row], s["q_pe"].to(dtype)[row]], -1)
    sc = torch.matmul(y.flatten(1, 2), torch.cat([c, k], -1).transpose(1, 2)).view(*y.shape[:3], -1).mul_(SCALE)
    t = torch.arange(sc.shape[-1], device="cuda")
    lens = s["seq_lens"].long()
    hidden = t[None, None, :] > (lens - n)[:, None, None] + i[None, :, None]
    sc.masked_fill_(hidden[:, :, None, :], -math.inf)
    return sc, t[None, :] < lens[:, None]


def _plain_mass(s):
    sc, real = _scores(s, torch.float32)
    rows = _real_rows(s)
    lse = torch.full(sc.shape[:3], math.inf, device="cuda")
    lse[rows] = s["lse"]                                             # a padding row has no weight
    w = sc.sub_(lse[..., None]).exp_().sum((1, 2))
    ctx = s["ctx"] if s["counted"] is None else s["counted"]
    t = torch.arange(w.shape[1], device="cuda")
    slot = (s["table"].long().repeat_interleave(PAGE, 1) * PAGE + t % PAGE)[real]
    old = torch.where((t[None, :] < ctx[:, None])[real], s["mass"][slot] * s["decay"], torch.zeros_like(s["mass"][slot]))
    s["mass"][slot] = old + w[real]
    return s["mass"]


def _own_mass(s):
    import mla_latent_kv_append_gb300 as mla
    case = s["case"]
    if "cache" not in s:
        # what the program keeps between steps: the layer's handle and a workspace
        s["cache"] = mla.CacheLayer(s["num_pages"], *FORMATS[case["fmt"]], pool=s["pool"])
        s["ws"] = torch.empty(mla.mla_mass_workspace_bytes(case["batch"], s["n"], case["heads"], s["max_new"]), dtype=torch.uint8,
                              device="cuda")
    mla.mla_token_mass(s["cache"], s["q_lat"], s["q_pe"], s["lse"], s["table"], s["q_start"], s["seq_lens"], s["ws"], s["mass"],
                       max_new=s["max_new"], decay=s["decay"], counted=s["counted"])
    return s["mass"]


def _plain_select(s):
    case, lens, keep = s["case"], s["seq_lens"].long(), s["keep"].long()
    t = torch.arange(s["table"].shape[1] * PAGE, device="cuda")[None, :]
    m = s["mass"].view(-1, PAGE)[s["table"].clamp(min=0).long()].flatten(1)
    sinks = keep.clamp(max=case["sinks"])
    recent = torch.minimum(keep - sinks, torch.full_like(keep, case["recent"]))
    m = torch.where((t < sinks[:, None]) | (t >= (lens - recent)[:, None]), torch.full_like(m, math.inf), m)
    m = torch.where(t < lens[:, None], m, torch.full_like(m, -math.inf))
    order = torch.sort(m, dim=1, descending=True, stable=True).indices[:, : s["max_keep"]]
    j = torch.arange(s["max_keep"], device="cuda")[None, :]
    some = j < keep[:, None]
    kept = torch.where(some, order, torch.full_like(order, 1 << 40)).sort(1).values
    return {"kept": torch.where(some, kept, torch.full_like(kept, -1)).int(), "kept_lens": keep.int()}


def _own_select(s):
    import mla_latent_kv_append_gb300 as mla
    if "out" not in s:
        s["out"] = {"kept": torch.empty((s["case"]["batch"], s["max_keep"]), dtype=torch.int32, device="cuda"),
                    "kept_lens": torch.empty(s["case"]["batch"], dtype=torch.int32, device="cuda")}
    o = s["out"]
    mla.mla_select_tokens(s["mass"], s["table"], s["seq_lens"], s["keep"], o["kept"], o["kept_lens"], sinks=s["case"]["sinks"],
                          recent=s["case"]["recent"])
    return o


def _plain_pages(s):
    old, new, table, free = s["old"].long(), s["new"].long(), s["table"], s["free"]
    was, now = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    head, tail = s["free_range"][0].long(), s["free_range"][1].long()
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    if s["case"]["move"]:
        moves = new < old
        take = torch.where(moves, now, torch.zeros_like(now))
        first = head + torch.cumsum(take, 0) - take
        fresh = free[(first[:, None] + col).clamp(0, free.numel() - 1)]
        mine = moves[:, None] & (col < now[:, None])
        back = moves[:, None] & (col < was[:, None])
        out = torch.where(moves[:, None], torch.where(mine, fresh, torch.full_like(fresh, -1)), table)
        s["page_table"][s["req"].long()] = torch.where(mine, fresh, s["page_table"][s["req"].long()])
    else:
        take = torch.zeros_like(now)
        back = (col >= now[:, None]) & (col < was[:, None])
        out = torch.where(col < now[:, None], table, torch.full_like(table, -1))
    flat = back.flatten()
    to = head + take.sum() - flat.sum()
    at = to + torch.cumsum(flat, 0) - 1
    at = torch.where(flat, at, torch.full_like(at, free.numel()))
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, at, table.flatten())
    free.copy_(longer[:-1])
    return {"table": out, "page_table": s["page_table"], "free": free, "lens": s["new"].clone(),
            "free_range": torch.stack([to, tail]).int()}


def _own_pages(s):
    import mla_latent_kv_append_gb300 as mla
    if "out" not in s:
        s["out"] = {"table": torch.empty_like(s["table"]), "lens": torch.empty_like(s["new"]),
                    "free_range": torch.empty(2, dtype=torch.int32, device="cuda")}
    o = s["out"]
    mla.mla_release_pages(s["old"], s["new"], s["req"], s["table"], s["page_table"], s["free"], s["free_range"], s["num_pages"],
                          o["table"], o["lens"], o["free_range"], move=s["case"]["move"])
    return {"page_table": s["page_table"], "free": s["free"], **o}


def _plain_move(s):
    lf, kf = FORMATS[s["case"]["fmt"]]
    at = _layout(s["case"]["fmt"])
    blocks = s["pool"].view(-1, at["bytes"])
    kept, j = s["kept"].long(), torch.arange(s["kept"].shape[1], device="cuda")
    moves = ((s["lens"] < s["seq_lens"])[:, None] & (j[None, :] < s["lens"][:, None])).nonzero(as_tuple=True)
    kept = kept[moves]
    src = s["table"].long()[moves[0], kept // PAGE] * PAGE + kept % PAGE
    dst = s["dst"].long()[moves[0], moves[1] // PAGE] * PAGE + moves[1] % PAGE
    (bs, us), (bd, ud) = (src // BLOCK, src % BLOCK), (dst // BLOCK, dst % BLOCK)

    def rows(off, row, pos):
        v = blocks[:, off:off + BLOCK * row].unflatten(1, (BLOCK, row // 16, 16))
        v[bd[:, None], ud[:, None], pos[ud]] = v[bs[:, None], us[:, None], pos[us]]

    def field(off, groups):
        v = blocks[:, off:off + groups * BLOCK * 4].unflatten(1, (groups, BLOCK, 4))
        v[bd, :, ud] = v[bs, :, us]

    rows(0, at["row"], _chunk_pos(at["row"]))
    rows(at["kpe"], at["krow"], _chunk_pos(at["krow"], kf))
    if lf:
        field(at["scale"], 32)
        field(at["bound"], 1)
    if lf == 2:
        field(at["zero"], 32)
    if kf:
        field(at["kscale"], 8)
    s["mass"][dst] = s["mass"][src]
    return {"pool": s["pool"], "mass": s["mass"]}


def _own_move(s):
    import mla_latent_kv_append_gb300 as mla
    if "cache" not in s:
        s["cache"] = mla.CacheLayer(s["num_pages"], *FORMATS[s["case"]["fmt"]], pool=s["pool"])
    mla.mla_move_tokens(s["cache"], s["table"], s["seq_lens"], s["kept"], s["lens"], s["dst"], mass=s["mass"])
    return {"pool": s["pool"], "mass": s["mass"]}


# ---------------------------------------------------------------------------
# work and exact
# ---------------------------------------------------------------------------

def _token_bytes(fmt):
    """A token's codes, scales, zero-points and k_pe."""
    at = _layout(fmt)
    return (at["bytes"] - (4 * BLOCK if "bound" in at else 0)) // BLOCK


def work(case):
    if case["op"] == "verify":
        drafts, size = _draft_lens(case), 4 if case["dtype"] == "fp32" else 2
        # a row of the target's for every sequence, one of the draft's where there are drafts to reject
        rows = sum(1 if case["lookup"] or d == 0 else 2 for d in drafts)
        return {"bytes": rows * case["vocab"] * size + sum(drafts) * (8 + 2 * size) + 4 * case["batch"] * (case["drafts"] + 6),
                "flops": rows * case["vocab"]}
    if case["op"] == "mass":
        ctx, new = _mass_lens(case)
        tokens, h = sum(ctx) + sum(new), case["heads"]
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        return {"bytes": tokens * (_token_bytes(case["fmt"]) + 4 + (0 if case["fresh"] else 4)) + sum(new) * h * (4 * D_C + 2 * D_R + 4),
                "flops": pairs * h * 2 * (D_C + D_R)}
    if case["op"] == "select":
        lens, keep = _keep_lens(case)
        return {"bytes": 4 * (sum(lens) + sum(_pages(t) for t in lens) + case["batch"] * (max(keep) + 3)), "flops": sum(lens)}
    if case["op"] == "pages":
        old, new = _page_lens(case)
        short = [(o, n) for o, n in zip(old, new) if n < o]
        back = sum(_pages(o) - (0 if case["move"] else _pages(n)) for o, n in short)
        fresh = sum(_pages(n) for _, n in short) if case["move"] else 0
        return {"bytes": 4 * (sum(_pages(o) for o in old) + back + 2 * fresh + case["batch"] * (case["max_pages"] + 4)), "flops": 0}
    lens, keep = _keep_lens(case)
    moved = sum(k for k, t in zip(keep, lens) if k < t)
    bound = 0 if case["fmt"] == "bf16" else 4
    return {"bytes": moved * (2 * (_token_bytes(case["fmt"]) + bound + 4) + 4), "flops": 0}


def exact(case, seed):
    if case["op"] == "mass":
        return _exact_mass(prepare(case, seed))
    if case["op"] == "move":
        return _exact_move(prepare(case, seed))
    return None                           # whole numbers: they have to be equal


def _exact_mass(s):
    """Sequence by sequence, key by key from the definition."""
    out = s["mass"].double()
    ends, lens, ctx = s["q_start"].tolist(), s["seq_lens"].tolist(), s["ctx"].tolist()
    for b, length in enumerate(lens):
        c, k = (x[:length] for x in _read(s["pool"], s["case"]["fmt"], s["table"][b, : _pages(length)], torch.float64))
        got = torch.zeros(length, dtype=torch.float64, device="cuda")
        for i, r in enumerate(range(ends[b], ends[b + 1])):
            sees = length - (ends[b + 1] - ends[b]) + i + 1
            score = s["q_lat"][r].double() @ c[:sees].t() + s["q_pe"][r].double() @ k[:sees].t()
            got[:sees] += torch.exp(score * SCALE - s["lse"][r].double()[:, None]).sum(0)
        at = torch.arange(length, device="cuda")
        slot = s["table"][b].long()[at // PAGE] * PAGE + at % PAGE
        before = ctx[b] if s["counted"] is None else int(s["counted"][b])
        out[slot] = torch.where(at < before, out[slot] * s["decay"], torch.zeros_like(got)) + got
    return out


def _exact_move(s):
    mass = s["mass"].cpu().numpy().astype(np.float64)
    src, dst = s["table"].cpu().numpy().astype(np.int64), s["dst"].cpu().numpy().astype(np.int64)
    kept, lens, before = s["kept"].cpu().numpy(), s["lens"].tolist(), s["seq_lens"].tolist()
    new = mass.copy()
    for b, n in enumerate(lens):
        if n < before[b]:
            j, t = np.arange(n), kept[b, :n]
            new[dst[b, j // PAGE] * PAGE + j % PAGE] = mass[src[b, t // PAGE] * PAGE + t % PAGE]
    return {"pool": None, "mass": torch.from_numpy(new)}
