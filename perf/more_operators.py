"""Measured cases of a quantized key/value cache: rows of new positions written into it, positions read back, and the
attention of new positions over it, for single tokens, the verification of drafts, and prompts.

`run` computes each operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, calls the library.  `exact` states the same operators in 64 bits.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"q8_0": 8, "q4_0": 4}
CELL = 16                                                   # positions that lie together in a page
DEV = "cuda"


# ------------------------------------------------------------------ cases

def attention(n_req, past, new, heads, kv, dim, fmt, dtype, page=64, causal=1, window=0):
    return {"op": "attention", "n_req": n_req, "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1],
            "heads": heads, "kv": kv, "dim": dim, "fmt": fmt, "dtype": dtype, "page": page, "causal": causal, "window": window}


def write(n_req, past, new, kv, dim, fmt, dtype, page=64):
    return {"op": "write", "n_req": n_req, "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1],
            "heads": 4 * kv, "kv": kv, "dim": dim, "fmt": fmt, "dtype": dtype, "page": page}


def read(n_req, length, kv, dim, fmt, dtype, page=64):
    return {"op": "read", "n_req": n_req, "past_lo": 0, "past_hi": 0, "new_lo": length[0], "new_hi": length[1],
            "kv": kv, "dim": dim, "fmt": fmt, "dtype": dtype, "page": page}


def listed():
    return [
        # one token of one request behind a short conversation: latency
        dict(attention(1, (700, 700), (1, 1), 32, 8, 128, "q4_0", "bf16"), name="attention 1 token, 700 positions"),
        # a decode batch of conversations of very different lengths
        dict(attention(64, (100, 8191), (1, 1), 32, 8, 128, "q4_0", "bf16"), name="attention 64 tokens, 100 to 8191 positions"),
        # one token of one request behind a whole book: the work of few heads spread over the GPU
        dict(attention(1, (131071, 131071), (1, 1), 32, 4, 128, "q8_0", "f16", page=256), name="attention 1 token, 131071 positions"),
        # a decode batch over one wide key/value head that all heads share, every request's whole cache visible
        dict(attention(24, (200, 6000), (1, 1), 16, 1, 256, "q8_0", "bf16", page=128, causal=0), name="attention 24 tokens, one wide head"),
        # the verify step of a batch: ragged drafts, small pages
        dict(attention(32, (500, 4000), (1, 8), 32, 4, 128, "q4_0", "bf16", page=16), name="attention 32 requests of 1 to 8 tokens"),
        # a verify step kept in 32 bits throughout, the model looks back a window of positions only
        dict(attention(9, (30, 1500), (1, 5), 16, 8, 64, "q8_0", "f32", page=32, window=512), name="attention 9 requests f32, window"),
        # a prompt with nothing before it
        dict(attention(1, (0, 0), (2011, 2011), 32, 8, 128, "q8_0", "bf16"), name="attention prompt of 2011 tokens"),
        # the fourth part of a long prompt: the largest
        dict(attention(1, (12289, 12289), (4096, 4096), 32, 8, 128, "q4_0", "f16"), name="attention 4096 tokens behind 12289"),
        # a decode batch's new rows, written and read back as the step after sees them
        dict(write(64, (100, 8191), (1, 1), 8, 128, "q4_0", "bf16"), name="write 64 tokens"),
        # three prompts
        dict(write(3, (0, 50), (1000, 4001), 8, 128, "q8_0", "f16"), name="write 3 prompts"),
        # a short request's cache taken out, to move it elsewhere
        dict(read(1, (333, 333), 8, 128, "q4_0", "bf16"), name="read 333 positions"),
        # a batch's caches taken out
        dict(read(16, (500, 8191), 8, 128, "q8_0", "bf16"), name="read 16 requests"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "attention", "write", "read"])
    largest = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        kv, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
        fmt, dtype = rng.choice(["q8_0", "q4_0"]), rng.choice(["f32", "f16", "bf16", "bf16"])
        page = rng.choice([16, 32, 64, 128, 256])
        if op == "attention":
            many = rng.random() < 0.35                      # prompts, else single tokens and drafts
            hi = _log(rng, 1, 131072 if not many else 16384)
            n = _log(rng, 9, 4096) if many else rng.randint(1, 8)
            c = attention(_log(rng, 1, 4 if many else 96), (_log(rng, 1, hi) - 1, hi), (rng.randint(1, n), n),
                          kv * rng.choice([1, 2, 4, 4, 7, 8]), kv, dim, fmt, dtype, page, int(rng.random() < 0.85),
                          0)
            if c["causal"] and rng.random() < 0.25:
                c["window"] = _log(rng, 1, 8192)
        elif op == "write":
            n = rng.choice([1, _log(rng, 1, 4000)])
            c = write(_log(rng, 1, 96), (0, _log(rng, 1, 4000)), (rng.randint(1, n), n), kv, dim, fmt, dtype, page)
        else:
            hi = _log(rng, 1, 8192)
            c = read(_log(rng, 1, 32), (rng.randint(1, hi), hi), kv, dim, fmt, dtype, page)
        # what a state holds stays within a few GB
        if _cost(c) <= largest and c["n_req"] * (c["past_hi"] + c["new_hi"]) * kv * dim <= 600e6:
            return c


def _cost(c):
    w = work(c)
    times = 16 if c["dtype"] == "f32" and c["op"] == "attention" else 1
    return max(w["bytes"] / 6.8e12, times * w["flops"] / 1.9e15)


@functools.lru_cache(maxsize=64)
def _lengths(n_req, past_lo, past_hi, new_lo, new_hi):
    """Of each request the positions before its new tokens, and the new tokens: the case's, not the seed's."""
    out = []
    for r in range(n_req):
        u = (((r + 1) * 2654435761 >> 8) & 0xFFFF) / 65536
        v = (((r + 1) * 2246822519 >> 9) & 0xFFFF) / 65536
        past = int(round((past_lo + 1) * ((past_hi + 1) / (past_lo + 1)) ** u)) - 1 if n_req > 1 else past_hi
        out.append((past, new_lo + int(v * (new_hi - new_lo + 1)) if n_req > 1 else new_hi))
    return out


def _requests(c):
    return _lengths(c["n_req"], c["past_lo"], c["past_hi"], c["new_lo"], c["new_hi"])


def work(case):
    c, e = case, 2 if case["dtype"] != "f32" else 4
    new = sum(n for _, n in _requests(c))
    row = c["kv"] * c["dim"]                                # values of a position's keys, or of its values
    stored = 2 * row // 32 * (2 + 4 * BITS[c["fmt"]])
    if c["op"] == "write":                                  # in, stored, read again, out
        return {"bytes": new * (4 * row * e + 2 * stored), "flops": 8 * new * row}
    if c["op"] == "read":
        return {"bytes": new * (2 * row * e + stored), "flops": 2 * new * row}
    seen = pairs = 0
    for past, n in _requests(c):
        first = [max(0, past + i + 1 - c["window"]) if c["window"] else 0 for i in (0, n - 1)]
        seen += past + n - first[0]
        for i in range(n):
            last = past + i + 1 if c["causal"] else past + n
            pairs += last - (max(0, last - c["window"]) if c["window"] else 0)
    return {"bytes": 2 * new * c["heads"] * c["dim"] * e + seen * stored, "flops": 4 * pairs * c["heads"] * c["dim"]}


# ------------------------------------------------------------------ the cache in memory
#
# A page holds `page` positions of all key/value heads: [kv][page / 16] cells of 16 positions.  A cell: the quants of its
# keys, of its values, the keys' scales [16][dim / 32], the values' scales [8][dim / 32][2].  Quants are stored unsigned
# (q + 128, or n).  A key's row is [unit][4][unit bytes]: lane c of 4 holds elements 8 c .. 8 c + 7 of every block of 32; a
# pair of positions' values is [unit][8][unit bytes]: lane g of 8 holds elements g, 8 + g, 16 + g and 24 + g of every block.

@functools.lru_cache(maxsize=16)
def _tables(fmt, dim):
    """Of each byte of a key's row and of a position's values: the elements in it ([bytes][1 or 2]), and its
    place in the cell for each of the 16 positions ([16][bytes])."""
    bits = BITS[fmt]
    rb = dim * bits // 8
    lane = rb // 4                                          # bytes of a lane, key row or pair of values
    ub = min(16, lane)
    ke, kp, ve, vp = [], [], [], []
    for r in range(rb):
        u, c, i = r // (4 * ub), r // ub % 4, r % ub
        w, y = (u * ub + i) // 4, i % 4
        if bits == 4:
            ke.append([32 * w + 8 * c + (2 * p if p < 4 else 2 * p - 7) for p in (2 * y, 2 * y + 1)])
        else:
            ke.append([32 * (w // 2) + 8 * c + 4 * (w % 2) + y])
        kp.append(r)
    for r in range(rb):
        u, g, i = r // (4 * ub), r // (ub // 2) % 8, r % (ub // 2)
        w, y = (u * ub + 2 * i) // 4, i % 2
        if bits == 4:
            ve.append([32 * w + 8 * j + g for j in (2 * y, 2 * y + 1)])
        else:
            ve.append([32 * (w // 2) + 8 * (2 * (w % 2) + y) + g])
        vp.append(u * 8 * ub + g * ub + (2 * i // 4) * 4 + y)
    pos = torch.arange(CELL)[:, None]
    kp, vp = torch.tensor(kp)[None] + pos * rb, torch.tensor(vp)[None] + 16 * rb + pos // 2 * (2 * rb) + pos % 2 * 2
    s = torch.arange(dim // 32 * 2)[None]                   # bytes of a position's scales
    ks = 32 * rb + pos * (dim // 16) + s
    vs = 32 * rb + dim + pos // 2 * (dim // 8) + s // 2 * 4 + pos % 2 * 2 + s % 2
    return torch.tensor(ke, device=DEV), torch.tensor(ve, device=DEV), torch.cat([kp, ks, vp, vs], 1).to(DEV)


def _cell_bytes(c):
    return 32 * (c["dim"] * BITS[c["fmt"]] // 8 + c["dim"] // 16)


def _codes(x, fmt):
    """[..., dim] in 32 bits -> scales [..., dim / 32] fp16 and unsigned quants [..., dim] uint8."""
    w = x.unflatten(-1, (-1, 32))
    size = w.abs()
    top, first = size.max(-1, keepdim=True)
    if fmt == "q8_0":
        d = (top / 127).clamp(max=65504.0)
        z = w / torch.where(d == 0, 1.0, d)
        q = ((z.abs() + 0.5).floor() * z.sign()).clamp(-127, 127) + 128
        q = torch.where(d == 0, 128.0, q)
    else:
        place = torch.arange(32, device=x.device)
        first = torch.where(size == top, place, 32).amin(-1, keepdim=True)
        d = (w.gather(-1, first) / -8).clamp(-65504.0, 65504.0)
        q = torch.where(d == 0, 8.0, (w / torch.where(d == 0, 1.0, d) + 8.5).floor().clamp(0, 15))
    odd = ~torch.isfinite(w).all(-1, keepdim=True)
    d, q = torch.where(odd, math.nan, d), torch.where(odd, 128.0 if fmt == "q8_0" else 8.0, q)
    return d.squeeze(-1).half(), q.flatten(-2).to(torch.uint8)


def _rows(k, v, fmt):
    """Keys and values [..., dim] -> the bytes of their positions, in the order of the tables."""
    ke, ve, _ = _tables(fmt, k.shape[-1])
    out = []
    for x, e in ((k, ke), (v, ve)):
        d, q = _codes(x, fmt)
        q = q[..., e.flatten()].unflatten(-1, e.shape)
        out += [q[..., 0] if fmt == "q8_0" else q[..., 0] | (q[..., 1] << 4), d.view(torch.uint8)]
    return torch.cat(out, -1)


def _values(b, fmt, dim):
    """The inverse of _rows, in 32 bits."""
    ke, ve, _ = _tables(fmt, dim)
    rb, out = dim * BITS[fmt] // 8, []
    for x, e in ((b[..., :b.shape[-1] // 2], ke), (b[..., b.shape[-1] // 2:], ve)):
        d = x[..., rb:].contiguous().view(torch.float16).float()
        x = x[..., :rb]
        q = (x if fmt == "q8_0" else torch.stack([x & 15, x >> 4], -1).flatten(-2)).float() - (128 if fmt == "q8_0" else 8)
        place = torch.empty(dim, dtype=torch.int64, device=DEV)
        place[e.flatten()] = torch.arange(dim, device=DEV)
        out.append((q[..., place].unflatten(-1, (-1, 32)) * d[..., None]).flatten(-2))
    return out


def _where(s, request, position):
    """Places in the pool of positions [n] of requests [n]: [n][kv][bytes of a row]."""
    c = s["case"]
    cells, cb = c["page"] // CELL, _cell_bytes(c)
    page = s["table"].long()[request, position // c["page"]]
    head = torch.arange(c["kv"], device=DEV)
    cell = (page[:, None] * c["kv"] + head) * cells + (position % c["page"] // CELL)[:, None]
    return cell[..., None] * cb + _tables(c["fmt"], c["dim"])[2][position % CELL][:, None]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    c, g = case, _gen(seed)
    reqs = _requests(c)
    total = [p + n for p, n in reqs]
    need = [-(-t // c["page"]) for t in total]
    s = {"case": dict(c)}
    s["offsets"] = torch.tensor([0] + [n for _, n in reqs], device=DEV).cumsum(0).to(torch.int32)
    s["lengths"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    # pages in the order in which a server happened to hand them out, some of them nobody's
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.zeros((c["n_req"], max(need)), dtype=torch.int32, device=DEV)
    used = torch.arange(max(need), device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    s["table"][used] = order[:sum(need)]
    T = sum(n for _, n in reqs)
    # keys have some dimensions that are always large, as rotary keys do
    big = 1 + 4 * (torch.rand((c["kv"], c["dim"]), generator=g, device=DEV) < 0.04)
    if c["op"] != "read":
        # the rows of a projection: queries, keys and values of a token side by side
        x = torch.randn((T, c["heads"] + 2 * c["kv"], c["dim"]), generator=g, device=DEV)
        x[:, c["heads"]:c["heads"] + c["kv"]] *= big
        s["x"] = x.flatten(1).to(DTYPES[c["dtype"]])
    s["tokens"] = T
    # what no position has been written to is whatever the memory held
    cells = n_pages * c["kv"] * (c["page"] // CELL)
    s["pool"] = torch.randint(0, 256, (cells * _cell_bytes(c),), generator=g, device=DEV, dtype=torch.uint8)
    if c["op"] != "write":
        for r, t in enumerate(total):
            for p0 in range(0, t, 16384):
                at = torch.arange(p0, min(t, p0 + 16384), device=DEV)
                kv = torch.randn((2, len(at), c["kv"], c["dim"]), generator=g, device=DEV)
                s["pool"][_where(s, torch.full_like(at, r), at)] = _rows(kv[0] * big, kv[1], c["fmt"])
    return s


def _parts(s):
    """Views of the projection's rows: queries, keys, values."""
    c = s["case"]
    h, kv, d = c["heads"], c["kv"], c["dim"]
    x = s["x"].unflatten(1, (-1, d))
    return x[:, :h], x[:, h:h + kv], x[:, h + kv:]


# ------------------------------------------------------------------ the operators

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import quantized_weight_matvec_hq_gb300 as hq
    c = s["case"]
    fmt, dt = hq.FMT_CODES[c["fmt"]], hq.DTYPE_CODES[c["dtype"]]
    T, R, W = s["tokens"], c["n_req"], s["table"].shape[1]
    if c["op"] != "read":
        (q, k, v), width = _parts(s), s["x"].shape[1]
    if "pages" not in s:                                    # outputs and workspace, made once as a program does
        s["pages"] = s["pool"].numel() // hq.hq_cache_page_bytes(fmt, c["kv"], c["dim"], c["page"])
        if c["op"] == "attention":
            s["out"] = torch.empty((T, c["heads"], c["dim"]), dtype=DTYPES[c["dtype"]], device=DEV)
            n = hq.hq_cache_attention_workspace(fmt, c["page"], W, R, T, c["heads"], c["kv"], c["dim"], dt)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        else:
            s["k"], s["v"] = (torch.empty((T, c["kv"], c["dim"]), dtype=DTYPES[c["dtype"]], device=DEV) for _ in "kv")
    cache = (s["pool"], s["pages"], c["page"], s["table"], W, s["offsets"], s["lengths"], R, T)
    if c["op"] == "attention":
        hq.hq_cache_attention(fmt, q, width, *cache, c["heads"], c["kv"], c["dim"], 1 / math.sqrt(c["dim"]), c["causal"],
                              c["window"], s["out"], c["heads"] * c["dim"], dt, s["ws"], s["ws"].numel())
        return s["out"]
    if c["op"] == "write":
        hq.hq_cache_write(fmt, k, width, v, width, *cache, c["kv"], c["dim"], dt)
    hq.hq_cache_read(fmt, s["k"], c["kv"] * c["dim"], s["v"], c["kv"] * c["dim"], *cache, c["kv"], c["dim"], dt)
    return {"k": s["k"], "v": s["v"]}


def _plain(s):
    c = s["case"]
    t = DTYPES[c["dtype"]]
    off, lengths = s["offsets"].long(), s["lengths"].long()
    T = s["tokens"]
    if c["op"] != "attention":
        n = off[1:] - off[:-1]
        req = torch.repeat_interleave(torch.arange(c["n_req"], device=DEV), n, output_size=T)
        at = _where(s, req, (lengths - n - off[:-1])[req] + torch.arange(T, device=DEV))
        if c["op"] == "write":
            _, k, v = _parts(s)
            s["pool"][at] = _rows(k.float(), v.float(), c["fmt"])
        k, v = _values(s["pool"][at], c["fmt"], c["dim"])
        return {"k": k.to(t), "v": v.to(t)}
    q = _parts(s)[0].float()
    out = torch.empty((T, c["heads"], c["dim"]), dtype=t, device=DEV)
    G, first = c["heads"] // c["kv"], 0
    for r, (past, n) in enumerate(_requests(c)):            # lengths that a program on the host knows
        pos = torch.arange(past + n, device=DEV)
        k, v = _values(s["pool"][_where(s, torch.full_like(pos, r), pos)], c["fmt"], c["dim"])
        here = past + torch.arange(n, device=DEV)[:, None]
        hidden = torch.zeros((n, past + n), dtype=torch.bool, device=DEV)
        if c["causal"]:
            hidden |= pos[None] > here
        if c["window"]:
            hidden |= pos[None] <= here - c["window"]
        for h in range(c["kv"]):
            qh = q[first:first + n, h * G:(h + 1) * G].transpose(0, 1) / math.sqrt(c["dim"])
            z = (qh.reshape(G * n, -1) @ k[:, h].T).view(G, n, -1).masked_fill_(hidden, -math.inf)
            z = torch.exp(z - z.amax(-1, keepdim=True))
            o = (z.view(G * n, -1) @ v[:, h]).view(G, n, -1) / z.sum(-1, keepdim=True)
            out[first:first + n, h * G:(h + 1) * G] = o.transpose(0, 1).to(t)
        first += n
    return out


# ------------------------------------------------------------------ the same in 64 bits

def _exact_cache(s, r, length):
    """Keys and values [length][kv][dim] of a request, its pages taken apart by their shape."""
    c = s["case"]
    kv, dim, bits, cells = c["kv"], c["dim"], BITS[c["fmt"]], c["page"] // CELL
    nb, rb = dim // 32, dim * bits // 8
    lane = rb // 4
    units, ub = max(1, lane // 16), min(16, lane)
    pages = s["table"][r, :-(-length // c["page"])].long()
    p = s["pool"].view(-1, kv, cells, _cell_bytes(c))[pages]            # [pages][kv][cells][bytes]
    quants, scales = p[..., :32 * rb], p[..., 32 * rb:].contiguous().view(torch.float16).to(torch.float64)
    ks = scales[..., :16 * nb].unflatten(-1, (16, nb))
    vs = scales[..., 16 * nb:].unflatten(-1, (8, nb, 2)).transpose(-1, -2).flatten(-3, -2)
    # keys: [16][units][4][words of a unit][bytes]
    k = quants[..., :16 * rb].unflatten(-1, (16, units, 4, ub // 4, 4)).transpose(-4, -3).flatten(-3, -2)    # [16][4][words][4]
    v = quants[..., 16 * rb:].unflatten(-1, (8, units, 8, ub // 4, 2, 2)).movedim(-2, -5).movedim(-3, -2)
    # values: [8][2][units][words of a unit][8][2] -> [16][words][8][2]
    v = v.flatten(-4, -3).flatten(-5, -4)
    if bits == 4:
        k = torch.stack([k[..., :2], k[..., 2:]], -1)                   # a word's low and high halves hold even and odd elements
        k = torch.stack([k % 16, torch.div(k, 16, rounding_mode="floor")], -2).to(torch.int16) - 8      # [...][byte][nibble][odd]
        k = k.flatten(-3).transpose(-3, -2)                             # [16][words][4][8]
        v = torch.stack([v % 16, torch.div(v, 16, rounding_mode="floor")], -1).to(torch.int16) - 8      # [16][words][8][2][2]
        v = v.flatten(-2).transpose(-2, -1)                             # [16][words][j][g]
    else:
        k = (k.to(torch.int16) - 128).unflatten(-2, (nb, 2)).flatten(-2).transpose(-3, -2)              # [16][blocks][4][8]
        v = (v.to(torch.int16) - 128).unflatten(-3, (nb, 2)).transpose(-2, -1).flatten(-3, -2)          # [16][blocks][j][g]
    out = []
    for x, d in ((k, ks), (v, vs)):
        x = (x.flatten(-2).to(torch.float64) * d[..., None]).flatten(-2)                                # [pages][kv][cells][16][dim]
        out.append(x.flatten(2, 3).transpose(1, 2).flatten(0, 1)[:length])
    return out


def _exact_stored(x, fmt):
    """Blocks by the definition: the quotient is one of 32-bit floats, which a 64-bit quotient rounded once to them is."""
    f32, f64 = torch.float32, torch.float64
    b = x.to(f64).unflatten(-1, (-1, 32))
    i = b.abs().argmax(-1, keepdim=True)
    m = b.gather(-1, (b.abs() == b.abs().gather(-1, i)).to(torch.uint8).argmax(-1, keepdim=True))
    d = (m.abs() / 127 if fmt == "q8_0" else m / -8).to(f32).to(f64)
    z = torch.where(d == 0, 0.0, (b / torch.where(d == 0, 1.0, d)).to(f32).to(f64))
    if fmt == "q8_0":
        q = torch.where(z < 0, -torch.floor(0.5 - z), torch.floor(z + 0.5)).clamp(-127, 127)
    else:
        q = torch.floor((z + 8.5).to(f32).to(f64)).clamp(0, 15) - 8
    return (q * d.to(torch.float16).to(f64)).flatten(-2)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "write":
        _, k, v = _parts(s)
        return {"k": _exact_stored(k, c["fmt"]), "v": _exact_stored(v, c["fmt"])}
    if c["op"] == "read":
        both = [_exact_cache(s, r, n) for r, (_, n) in enumerate(_requests(c))]
        return {"k": torch.cat([k for k, _ in both]), "v": torch.cat([v for _, v in both])}
    q, outs = _parts(s)[0].to(torch.float64), []
    for past, n in _requests(c):
        k, v = _exact_cache(s, len(outs), past + n)
        at = sum(len(o) for o in outs)
        o = torch.empty((n, c["heads"], c["dim"]), dtype=torch.float64, device=DEV)
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            row = torch.arange(past + i0, past + i1, device=DEV)
            far = row[:, None] - torch.arange(past + n, device=DEV)[None]
            see = torch.ones_like(far, dtype=torch.bool)
            if c["causal"]:
                see = far >= 0
            if c["window"]:
                see = see & (far < c["window"])
            for h in range(c["heads"]):
                g = h // (c["heads"] // c["kv"])
                z = (q[at + i0:at + i1, h] @ k[:, g].T) * c["dim"] ** -0.5
                o[i0:i1, h] = torch.softmax(torch.where(see, z, -math.inf), -1) @ v[:, g]
        outs.append(o)
    return torch.cat(outs)
