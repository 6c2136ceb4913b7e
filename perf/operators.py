"""The serving-step operators around the paged latent cache, and their plain forms.

Three operators that a step of chunked serving runs one after the other:

* plan:  block tables, slot map, positions and lengths of a step, from the
  requests' lengths and a list of free pages (whole numbers);
* rope:  rotary positions on the RoPE parts of the queries and keys, one or
  several position axes, either pair layout, forward or inverse;
* chunk: causal attention of every sequence's new tokens over the paged,
  quantized latent cache, from the projected query to the per-head output.

A case is a dict of plain values; sequence lengths follow from its own
``lens_seed``, every tensor's values from the seed that prepare() gets.
"""

import math
import random

import torch

own = False

D_C, D_R, D_N, D_V, PAGE, BLOCK = 512, 64, 128, 128, 64, 32
SCALE = 1.0 / math.sqrt(D_N + D_R)

# (latent format, k_pe format) of a cache -> the library's format numbers
FORMATS = {"bf16": (0, 0), "int8": (1, 1), "int4": (2, 1), "int4_int4": (2, 3)}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one chat request being decoded: the step's plan is pure latency
        {"name": "plan_one", "op": "plan", "batch": 1, "rows": 16, "max_pages": 64, "chunks": 0, "chunk": 0,
         "ctx_lo": 100, "ctx_hi": 4000, "pad": 0, "lens_seed": 1},
        # a busy server: 256 requests, most decoding, eight of them prefilling a chunk
        {"name": "plan_busy", "op": "plan", "batch": 256, "rows": 512, "max_pages": 512, "chunks": 8, "chunk": 777,
         "ctx_lo": 1, "ctx_hi": 32000, "pad": 33, "lens_seed": 2},
        # an offline batch at the library's batch limit, a few short chunks each
        {"name": "plan_offline", "op": "plan", "batch": 4096, "rows": 5000, "max_pages": 640, "chunks": 4000, "chunk": 16,
         "ctx_lo": 1, "ctx_hi": 40000, "pad": 0, "lens_seed": 3},
        # eight requests decoding at far positions
        {"name": "rope_decode", "op": "rope", "n": 8, "heads": 16, "axes": 1, "interleaved": True, "inverse": False,
         "far": 163840, "amp": 1.0},
        # a prefill chunk of images and text: time, height and width positions
        {"name": "rope_axes", "op": "rope", "n": 1999, "heads": 64, "axes": 3, "interleaved": False, "inverse": False,
         "far": 32768, "amp": 1.0},
        # a long prefill at the most heads, with a long-context frequency table; the inverse is its gradient
        {"name": "rope_long_inverse", "op": "rope", "n": 8192, "heads": 128, "axes": 1, "interleaved": True,
         "inverse": True, "far": 1048576, "amp": 1.1},
        # one request's decode token: latency
        {"name": "chunk_decode_one", "op": "chunk", "fmt": "int8", "heads": 16, "batch": 1, "ctx_lo": 4096, "ctx_hi": 4096,
         "new": 1, "chunks": 0, "chunk": 0, "lens_seed": 4},
        # a decode batch of long contexts in the smallest format
        {"name": "chunk_decode_long", "op": "chunk", "fmt": "int4_int4", "heads": 16, "batch": 32, "ctx_lo": 32767,
         "ctx_hi": 32767, "new": 1, "chunks": 0, "chunk": 0, "lens_seed": 5},
        # speculative decoding: up to five drafted tokens are checked per sequence, ragged
        {"name": "chunk_verify", "op": "chunk", "fmt": "bf16", "heads": 64, "batch": 24, "ctx_lo": 1000, "ctx_hi": 16000,
         "new": 5, "chunks": 0, "chunk": 0, "lens_seed": 6},
        # continuous batching: two prefill chunks ride along with decoding requests
        {"name": "chunk_mixed", "op": "chunk", "fmt": "int8", "heads": 16, "batch": 40, "ctx_lo": 60, "ctx_hi": 12000,
         "new": 2, "chunks": 2, "chunk": 1023, "lens_seed": 7},
        # a 2048-token chunk after 32768 cached tokens
        {"name": "chunk_after_long", "op": "chunk", "fmt": "int4", "heads": 16, "batch": 1, "ctx_lo": 32768, "ctx_hi": 32768,
         "new": 0, "chunks": 1, "chunk": 2048, "lens_seed": 8},
        # the first 8192 tokens of a prompt at 64 heads
        {"name": "chunk_prompt", "op": "chunk", "fmt": "int8", "heads": 64, "batch": 1, "ctx_lo": 0, "ctx_hi": 0,
         "new": 0, "chunks": 1, "chunk": 8192, "lens_seed": 9},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "chunk", "chunk"])
    if op == "plan":
        batch = _log_int(rng, 1, 4096)
        chunks = rng.randint(0, batch)
        return {"op": op, "batch": batch, "rows": batch + rng.randint(0, 1000), "max_pages": _log_int(rng, 32, 640),
                "chunks": chunks, "chunk": _log_int(rng, 1, max(1, min(2000, 65536 // max(1, chunks)))),
                "ctx_lo": 1, "ctx_hi": _log_int(rng, 64, 38000), "pad": rng.randint(0, 64), "lens_seed": rng.randint(0, 1 << 30)}
    if op == "rope":
        return {"op": op, "n": _log_int(rng, 1, 8192), "heads": rng.choice([16, 32, 48, 64, 128]), "axes": rng.randint(1, 4),
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5, "far": _log_int(rng, 1024, 1 << 22),
                "amp": rng.choice([1.0, round(rng.uniform(0.7, 1.4), 3)])}
    fmt, heads = rng.choice(sorted(FORMATS)), rng.choice([16, 32, 48, 64, 128])
    for _ in range(1000):
        kind = rng.choice(["decode", "verify", "mixed", "prefill"])
        case = {"op": op, "fmt": fmt, "heads": heads, "batch": 1, "ctx_lo": 0, "ctx_hi": 0, "new": 0, "chunks": 0, "chunk": 0,
                "lens_seed": rng.randint(0, 1 << 30)}
        case["ctx_hi"] = _log_int(rng, 16, 65536)
        case["ctx_lo"] = rng.randint(0, case["ctx_hi"])
        if kind == "decode":
            case |= {"batch": _log_int(rng, 1, 200), "new": 1}
        elif kind == "verify":
            case |= {"batch": _log_int(rng, 1, 64), "new": rng.randint(2, 40)}
        elif kind == "mixed":
            case |= {"batch": _log_int(rng, 4, 64), "new": rng.randint(1, 4), "chunks": rng.randint(1, 3), "chunk": _log_int(rng, 65, 2500)}
        else:
            case |= {"batch": rng.randint(1, 3), "chunk": _log_int(rng, 65, 8000)}
            case["chunks"] = case["batch"]
        ctx, new = _chunk_lens(case)
        if work(case)["flops"] <= 1.4e12 and sum(ctx) + sum(new) <= 1_200_000 and sum(new) * heads <= 600_000:
            return case
    raise RuntimeError("no case within the limits")


def _chunk_lens(case):
    """(cached tokens, new tokens) of every sequence: `chunks` sequences have a
    chunk of about `chunk` tokens (the first exactly), the others 1 .. `new`."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["ctx_lo"], case["ctx_hi"]
    ctx = [hi if lo == hi else int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) for _ in range(case["batch"])]
    new = []
    for b in range(case["batch"]):
        if b < case["chunks"]:
            new.append(case["chunk"] if b == 0 else r.randint(max(1, case["chunk"] // 2), case["chunk"]))
        else:
            new.append(r.randint(1, max(1, case["new"])))
    both = list(zip(ctx, new))
    r.shuffle(both)
    return [c for c, _ in both], [n for _, n in both]


def _plan_lens(case):
    r = random.Random(case["lens_seed"])
    cap = case["max_pages"] * PAGE
    ctx, new = [], []
    for b in range(case["batch"]):
        n = r.randint(1, case["chunk"]) if b < case["chunks"] and case["chunk"] else r.choice([1, 1, 1, 1, 1, 1, 1, 0])
        n = min(n, cap)
        c = int(math.exp(r.uniform(math.log(case["ctx_lo"]), math.log(case["ctx_hi"] + 1))))
        ctx.append(min(c, cap - n))
        new.append(n)
    both = list(zip(ctx, new))
    r.shuffle(both)
    return [c for c, _ in both], [n for _, n in both]


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
    """uint8 [..., chunks, 16] -> float32 [..., chunks * 32] nibble values in channel order."""
    w = chunks.reshape(*chunks.shape[:-1], 4, 4)
    n = torch.stack([w & 15, w >> 4], dim=-1).reshape(*chunks.shape[:-1], 32)      # word j, nibble k at 8 j + k
    ch = _nibble_channels(chunks.device)
    out = torch.empty_like(n)
    out[..., ch] = n
    return out.reshape(*chunks.shape[:-2], -1).float()


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


# ---------------------------------------------------------------------------
# prepare
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return {"plan": _prepare_plan, "rope": _prepare_rope, "chunk": _prepare_chunk}[case["op"]](case, g, seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, g, seed):
    ctx, new = _plan_lens(case)
    old = [_pages(c) for c in ctx]
    need = sum(_pages(c + n) for c, n in zip(ctx, new)) - sum(old)
    num_pages = sum(old) + need + 1000
    perm = torch.randperm(num_pages, generator=g, device="cuda").int()
    rows = torch.randperm(case["rows"], generator=g, device="cuda")[: case["batch"]].int()
    table = torch.full((case["rows"], case["max_pages"]), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(case["max_pages"], device="cuda")[None, :] < _ints(old)[:, None]
    full = torch.full((case["batch"], case["max_pages"]), -1, dtype=torch.int32, device="cuda")
    full[used] = perm[: sum(old)]
    table[rows.long()] = full
    free, head = perm[sum(old):].contiguous(), 37
    free = torch.cat([free[:head].flip(0), free[head:]]).contiguous()
    return {"case": case, "ctx": _ints(ctx), "new": _ints(new), "req": rows, "table": table, "free": free,
            "free_range": _ints([head, free.numel()]), "n": sum(new) + case["pad"], "num_pages": num_pages}


def _prepare_rope(case, g, seed):
    n, h = case["n"], case["heads"]
    q = torch.randn((n, h, D_N + D_R), generator=g, device="cuda").bfloat16()
    kv = torch.randn((n, D_C + D_R), generator=g, device="cuda").bfloat16()
    first = torch.randint(0, case["far"], (case["axes"], 1), generator=g, device="cuda")
    pos = (first + torch.arange(n, device="cuda")[None, :] // torch.tensor([1, 4, 1, 2], device="cuda")[: case["axes"], None]).int()
    f = 10000.0 ** (-torch.arange(0, D_R, 2, dtype=torch.float64) / D_R)
    # a long-context table: the low frequencies are interpolated by 40
    ramp = ((torch.arange(D_R // 2, dtype=torch.float64) - 10) / 13).clamp(0, 1)
    f = f * (1 - ramp) + f / 40 * ramp if case["far"] > 100000 else f
    per = {1: [32], 2: [12, 20], 3: [8, 12, 12], 4: [5, 9, 9, 9]}[case["axes"]]
    return {"case": case, "q": q, "kv": kv, "pos": pos.contiguous(), "inv_freq": f.float().cuda(),
            "axis": [a for a, m in enumerate(per) for _ in range(m)]}


def _prepare_chunk(case, g, seed):
    ctx, new = _chunk_lens(case)
    n, h, lens = sum(new), case["heads"], [c + m for c, m in zip(ctx, new)]
    pages = [_pages(t) for t in lens]
    at = _layout(case["fmt"])
    num_pages = sum(pages)
    perm = torch.randperm(num_pages, generator=g, device="cuda").int()
    max_pages = max(pages)
    table = torch.full((case["batch"], max_pages), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(max_pages, device="cuda")[None, :] < _ints(pages)[:, None]
    table[used] = perm
    # latents behind a norm: unit-sized channels of uneven gain, some far from zero, a few large ones
    gain = torch.exp(0.6 * torch.randn(D_C, generator=g, device="cuda"))
    mean = 0.5 * torch.randn(D_C, generator=g, device="cuda")
    gain[torch.randperm(D_C, generator=g, device="cuda")[:4]] *= 6
    pool = torch.zeros((num_pages, 2 * at["bytes"]), dtype=torch.uint8, device="cuda")
    step = 4096
    for p in range(0, num_pages, step):
        part = pool[p:p + step].view(-1, at["bytes"])
        c = (mean + gain * torch.randn((part.shape[0], BLOCK, D_C), generator=g, device="cuda")).bfloat16()
        k = torch.randn((part.shape[0], BLOCK, D_R), generator=g, device="cuda").bfloat16()
        _fill(part, case["fmt"], c, k)
    return {"case": case, "pool": pool.view(-1), "num_pages": num_pages, "table": table, "ctx": ctx, "new_lens": new,
            "q": torch.randn((n, h, D_N + D_R), generator=g, device="cuda").bfloat16(),
            "w_uk": (torch.randn((h, D_N, D_C), generator=g, device="cuda") / math.sqrt(D_C)).bfloat16(),
            "w_uv": (torch.randn((h, D_C, D_V), generator=g, device="cuda") / math.sqrt(D_C)).bfloat16(),
            "q_start": _ints([sum(new[:b]) for b in range(len(new) + 1)]), "seq_lens": _ints(lens)}


# ---------------------------------------------------------------------------
# run
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "chunk": _own_chunk}[op](state)
    return {"plan": _plain_plan, "rope": _plain_rope, "chunk": _plain_chunk}[op](state)


def _plain_plan(s):
    ctx, new, table = s["ctx"].long(), s["new"].long(), s["table"]
    old, now = (ctx + PAGE - 1) // PAGE, (ctx + new + PAGE - 1) // PAGE
    need = now - old
    head = s["free_range"][0].long()
    first = head + torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=ctx.device)[None, :]
    rows = table[s["req"].long()]
    fresh = (col >= old[:, None]) & (col < now[:, None])
    at = (first[:, None] + col - old[:, None]).clamp(0, s["free"].numel() - 1)
    rows = torch.where(fresh, s["free"][at], rows)
    table[s["req"].long()] = rows
    block_table = torch.where(col < now[:, None], rows, torch.full_like(rows, -1))
    q_end = torch.cumsum(new, 0)
    q_start = torch.cat([torch.zeros_like(q_end[:1]), q_end])
    i = torch.arange(s["n"], device=ctx.device)
    b = torch.searchsorted(q_end, i, right=True)
    real = b < ctx.numel()
    bb = b.clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[bb] + i - q_start[bb], torch.zeros_like(i))
    slot = torch.where(real, block_table[bb, pos // PAGE].long() * PAGE + pos % PAGE, torch.full_like(i, -1))
    token_req = torch.where(real, b, torch.full_like(b, -1))
    return {"table": table, "block_table": block_table, "q_start": q_start.int(), "seq_lens": (ctx + new).int(),
            "positions": pos.int(), "token_req": token_req.int(), "slot": slot.int(), "free_head": (head + need.sum()).int().view(1)}


def _own_plan(s):
    import mla_latent_kv_append_gb300 as mla
    if "out" not in s:
        b, n = s["ctx"].numel(), s["n"]
        e = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s["out"] = {"block_table": e(b, s["table"].shape[1]), "q_start": e(b + 1), "seq_lens": e(b), "positions": e(n),
                    "token_req": e(n), "slot": e(n), "free_head": e(1)}
    o = s["out"]
    mla.mla_plan_chunks(s["ctx"], s["new"], s["req"], s["table"], s["free"], s["free_range"], s["num_pages"],
                        o["block_table"], o["q_start"], o["seq_lens"], o["positions"], o["token_req"], o["slot"],
                        o["free_head"])
    return {"table": s["table"], **o}


def _plain_rope(s):
    case = s["case"]
    f = s["inv_freq"].double()
    ang = s["pos"].double()[s["axis"]].t() * f[None, :]                # [n, 32]: pair i turns with its own axis
    cos, sin = (ang.cos() * case["amp"]).float(), (ang.sin() * case["amp"]).float()
    sin = -sin if case["inverse"] else sin

    def turn(x):
        x = x.float()
        c, d = (cos, sin) if x.dim() == 2 else (cos[:, None], sin[:, None])
        if case["interleaved"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * c - b * d, a * d + b * c], -1).reshape(x.shape).bfloat16()
        a, b = x[..., : D_R // 2], x[..., D_R // 2:]
        return torch.cat([a * c - b * d, a * d + b * c], -1).bfloat16()

    return {"q_pe": turn(s["q"][..., D_N:]), "k_pe": turn(s["kv"][:, D_C:])}


def _own_rope(s):
    import mla_latent_kv_append_gb300 as mla
    case = s["case"]
    if "out" not in s:
        s["out"] = (torch.empty((case["n"], case["heads"], D_R), dtype=torch.bfloat16, device="cuda"),
                    torch.empty((case["n"], D_R), dtype=torch.bfloat16, device="cuda"))
    q_out, k_out = s["out"]
    mla.mla_rope(s["q"][..., D_N:], s["kv"][:, D_C:], s["pos"], s["inv_freq"], q_out, k_out, pair_axis=s["axis"],
                 interleaved=case["interleaved"], inverse=case["inverse"], amplitude=case["amp"])
    return {"q_pe": q_out, "k_pe": k_out}


def _costs(ctx, new):
    """Per head: (absorbed, expanded) flops of one sequence's attention, projections included."""
    pairs = new * ctx + new * (new + 1) // 2
    return (pairs * 2 * (D_C + D_R + D_C) + new * 2 * 2 * D_N * D_C,
            pairs * 2 * (D_N + D_R + D_V) + (ctx + new) * 2 * D_C * (D_N + D_V))


def _plain_chunk(s):
    """Sequences with the same number of new tokens go together, padded to the
    longest; each group takes the bracketing that needs fewer operations."""
    case = s["case"]
    q, w_uk, w_uv = s["q"].float(), s["w_uk"].float(), s["w_uv"].float()
    o = torch.empty((q.shape[0], case["heads"], D_V), dtype=torch.bfloat16, device=q.device)
    starts = [sum(s["new_lens"][:b]) for b in range(case["batch"])]
    for n in sorted(set(s["new_lens"])):
        members = [b for b in range(case["batch"]) if s["new_lens"][b] == n]
        lens = [s["ctx"][b] + n for b in members]
        # so many at a time that their scores and keys stay within a few GB
        per = max(1, int(4e9 // (4 * max(lens) * (n * case["heads"] + 2 * (D_C + D_R)))))
        for m in range(0, len(members), per):
            part = members[m:m + per]
            _plain_group(s, q, w_uk, w_uv, o, part, n, [starts[b] for b in part])
    return o


def _plain_group(s, q, w_uk, w_uv, o, part, n, starts):
    top = max(s["ctx"][b] for b in part) + n
    sel = torch.tensor(part, device=q.device)
    rows = torch.tensor(starts, device=q.device)[:, None] + torch.arange(n, device=q.device)[None, :]
    ctx = torch.tensor([s["ctx"][b] for b in part], device=q.device)
    pages = s["table"][sel, : _pages(top)].clamp(min=0)
    c, k = _read(s["pool"], s["case"]["fmt"], pages, torch.float32)      # [m, T, 512], [m, T, 64]
    t = torch.arange(c.shape[1], device=q.device)
    # [m, 1, n, T]: key t is behind the query at position ctx + i, or past the sequence's end
    hidden = t[None, None, None, :] > (ctx[:, None] + torch.arange(n, device=q.device)[None, :])[:, None, :, None]
    x = q[rows].transpose(1, 2)                                        # [m, H, n, 192]
    absorbed, expanded = _costs(top - n, n)
    few = absorbed <= expanded
    step = x.shape[1] if few else max(1, int(4e9 // (4 * n * c.shape[1] * len(part))))      # heads at a time
    for h0 in range(0, x.shape[1], step):
        h1 = min(x.shape[1], h0 + step)
        xn, xr = x[:, h0:h1, :, :D_N], x[:, h0:h1, :, D_N:]
        if few:
            y = torch.cat([torch.einsum("mhnd,hdc->mhnc", xn, w_uk[h0:h1]), xr], -1)
            p = torch.matmul(y.flatten(1, 2), torch.cat([c, k], -1).transpose(1, 2)).view(*y.shape[:3], -1)
        else:
            p = torch.matmul(xn, torch.einsum("mtc,hdc->mhdt", c, w_uk[h0:h1]))
            p += torch.matmul(xr.flatten(1, 2), k.transpose(1, 2)).view(p.shape)
        p.mul_(SCALE).masked_fill_(hidden, -math.inf)
        p.sub_(p.amax(-1, keepdim=True)).exp_()
        p.div_(p.sum(-1, keepdim=True))
        if few:
            lat = torch.matmul(p.flatten(1, 2), c).view(*p.shape[:3], D_C)
            y = torch.einsum("mhnc,hcv->mhnv", lat, w_uv[h0:h1])
        else:
            y = torch.matmul(p, torch.einsum("mtc,hcv->mhtv", c, w_uv[h0:h1]))
        o[rows, h0:h1] = y.transpose(1, 2).bfloat16()


def _own_chunk(s):
    import mla_latent_kv_append_gb300 as mla
    case = s["case"]
    if "cache" not in s:
        # what the program keeps between steps: the layer's handle, a workspace and the output buffer
        s["cache"] = mla.CacheLayer(s["num_pages"], *FORMATS[case["fmt"]], pool=s["pool"])
        s["max_new"] = max(s["new_lens"])
        s["kv_tokens"] = sum((c + n + 127) // 128 * 128 for c, n in zip(s["ctx"], s["new_lens"]) if n > mla.CHUNK_SHORT)
        s["ws"] = torch.empty(mla.mla_chunk_workspace_bytes(case["batch"], s["q"].shape[0], case["heads"], s["max_new"],
                                                            s["kv_tokens"]), dtype=torch.uint8, device="cuda")
        s["o"] = torch.empty((s["q"].shape[0], case["heads"], D_V), dtype=torch.bfloat16, device="cuda")
    q = s["q"]
    mla.mla_chunk_attention(s["cache"], q[..., :D_N], q[..., D_N:], s["w_uk"], s["w_uv"], s["table"], s["q_start"],
                            s["seq_lens"], s["ws"], s["o"], max_new=s["max_new"], kv_tokens=s["kv_tokens"])
    return s["o"]


# ---------------------------------------------------------------------------
# work and exact
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "plan":
        ctx, new = _plan_lens(case)
        used = sum(_pages(c) for c in ctx)
        fresh = sum(_pages(c + n) for c, n in zip(ctx, new)) - used
        words = 3 * case["batch"] + used + fresh + fresh + case["batch"] * case["max_pages"] + 2 * case["batch"]
        return {"bytes": 4 * (words + 3 * (sum(new) + case["pad"])), "flops": 0}
    if case["op"] == "rope":
        n, h = case["n"], case["heads"]
        return {"bytes": 2 * 2 * n * (h + 1) * D_R + 4 * n * case["axes"], "flops": 3 * n * (h + 1) * D_R}
    ctx, new = _chunk_lens(case)
    h, tok = case["heads"], sum(ctx) + sum(new)
    at = _layout(case["fmt"])
    kept = at["bytes"] - (4 * BLOCK if "bound" in at else 0)
    # weights: what the chosen bracketing multiplies by, once
    return {"bytes": tok * kept // BLOCK + sum(new) * h * 2 * (D_N + D_R + D_V) + h * 2 * D_C * (D_N + D_V),
            "flops": h * sum(min(_costs(c, n)) for c, n in zip(ctx, new))}


def exact(case, seed):
    if case["op"] == "plan":
        return None                       # whole numbers: they have to be equal
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_chunk(s)


def _exact_rope(s):
    case = s["case"]
    turn = torch.zeros((case["n"], D_R // 2), dtype=torch.complex128, device="cuda")
    for i, a in enumerate(s["axis"]):
        t = s["pos"][a].double() * s["inv_freq"][i].double()
        turn[:, i] = torch.polar(torch.full_like(t, case["amp"]), -t if case["inverse"] else t)

    def apply(x):
        x = x.double()
        z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) if case["interleaved"] \
            else torch.complex(x[..., : D_R // 2].contiguous(), x[..., D_R // 2:].contiguous())
        z = z * (turn if x.dim() == 2 else turn[:, None])
        return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)

    return {"q_pe": apply(s["q"][..., D_N:]), "k_pe": apply(s["kv"][:, D_C:])}


def _exact_chunk(s):
    """Sequence by sequence and head by head: per-head keys and values where a
    sequence has many new tokens, absorbed queries where it has few."""
    case = s["case"]
    if sum(min(_costs(c, n)) for c, n in zip(s["ctx"], s["new_lens"])) * case["heads"] > 6e12:
        return None
    out = torch.empty((s["q"].shape[0], case["heads"], D_V), dtype=torch.float64, device="cuda")
    row = 0
    for b, (ctx, n) in enumerate(zip(s["ctx"], s["new_lens"])):
        t = ctx + n
        c, k = (x[:t] for x in _read(s["pool"], case["fmt"], s["table"][b, : _pages(t)], torch.float64))
        seen = torch.ones((n, t), dtype=torch.bool, device="cuda").tril(ctx)
        q = s["q"][row:row + n].double()
        group = max(1, min(case["heads"], int(8e8 // (n * t + t * 256))))
        for h0 in range(0, case["heads"], group):
            h = slice(h0, min(h0 + group, case["heads"]))
            qn, qr = q[:, h, :D_N].permute(1, 0, 2), q[:, h, D_N:].permute(1, 0, 2)
            uk, uv = s["w_uk"][h].double(), s["w_uv"][h].double()
            if n <= 100:
                sc = (qn @ uk) @ c.t() + qr @ k.t()
            else:
                sc = qn @ (uk @ c.t()) + qr @ k.t()
            p = torch.softmax((sc * SCALE).masked_fill(~seen, -math.inf), -1)
            v = (p @ c) @ uv if n <= 100 else p @ (c @ uv)
            out[row:row + n, h] = v.permute(1, 0, 2)
        row += n
    return out
