"""Measured cases of the batched speculative step: the products of many tokens with quantized weights (grouped by
expert, or shared with an adapter per request), the probabilities of the logits, and the verification of drafts.

`run` computes each operator in its plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where `own` is true, calls the library.  `exact` states the same operators in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK_BYTES = {"q8_0": 34, "q4_0": 18}
DEV = "cuda"


# ------------------------------------------------------------------ cases

def moe(n_tokens, rows, cols, dtype, epilogue, per_slot=0, n_experts=128, n_active=8, skew=0.0):
    return {"op": "moe", "n_tokens": n_tokens, "rows": rows, "cols": cols, "dtype": dtype, "epilogue": epilogue,
            "per_slot": per_slot, "n_experts": n_experts, "n_active": n_active, "skew": skew}


def lora(n_tokens, rows, cols, dtype, fmt="q8_0", rank=16, n_adapters=8, n_req=1, bare=0.0):
    return {"op": "lora", "n_tokens": n_tokens, "rows": rows, "cols": cols, "dtype": dtype, "fmt": fmt, "rank": rank,
            "n_adapters": n_adapters, "n_req": n_req, "bare": bare}


def softmax(n_rows, vocab, dtype, warm=1):
    return {"op": "softmax", "n_rows": n_rows, "vocab": vocab, "dtype": dtype, "warm": warm}


def verify(n_req, most, vocab, sure=0):
    return {"op": "verify", "n_req": n_req, "most": most, "vocab": vocab, "sure": sure}


def listed():
    return [
        # one request's verify of five tokens through an expert layer's gate|up matrices: latency and weight bytes
        dict(moe(5, 1536, 2048, "bf16", "swiglu"), name="moe gate|up 5 tokens"),
        # a short prompt's down projection with the router's weighted sum; ragged groups of about 32 tokens
        dict(moe(517, 2048, 768, "bf16", "combine", per_slot=1, skew=0.5), name="moe down 517 tokens"),
        # a batch kept in 32 bits throughout, as the decode calls do
        dict(moe(131, 1536, 2048, "f32", "none"), name="moe 131 tokens f32"),
        # a long prompt: the largest grouped product
        dict(moe(4096, 1536, 2048, "bf16", "swiglu", skew=0.5), name="moe gate|up 4096 tokens"),
        # one token of one request with an adapter beside the output projection: latency
        dict(lora(1, 4096, 4096, "bf16", n_req=1), name="adapters o 1 token"),
        # a decode batch, every request with an adapter of its own or none, beside the widest projection
        dict(lora(64, 28672, 4096, "bf16", n_adapters=48, n_req=64, bare=0.1), name="adapters gate|up 64 tokens"),
        # a 4-bit base kept in 32 bits: the down projection of several requests' verifies
        dict(lora(45, 4096, 14336, "f32", fmt="q4_0", rank=8, n_req=9), name="adapters down 45 tokens q4_0"),
        # prompts of nine requests at once
        dict(lora(2011, 6144, 4096, "f16", rank=64, n_req=9), name="adapters q|k|v 2011 tokens"),
        # one request's verify rows, logits as a 16-bit head leaves them
        dict(softmax(5, 151936, "bf16"), name="softmax 5 rows"),
        # the verify rows of 64 requests
        dict(softmax(512, 128256, "f32"), name="softmax 512 rows"),
        # one request, four drafts
        dict(verify(1, 4, 151936), name="verify 1 request"),
        # 64 requests with 0 to 7 drafts each
        dict(verify(64, 7, 128256), name="verify 64 requests"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "lora", "lora", "softmax", "verify"])
    largest = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "moe":
            epi = rng.choice(["none", "swiglu", "combine"])
            rows = _log(rng, 8, 2048)
            E = rng.choice([8, 16, 61, 128])
            c = moe(_log(rng, 1, 4096), rows + (rows & 1 if epi == "swiglu" else 0), 256 * rng.randint(1, 8),
                    rng.choice(["f32", "f16", "bf16", "bf16"]), epi, rng.randint(0, 1), E,
                    rng.randint(1, 8), rng.choice([0.0, 0.5, 1.5]))
        elif op == "lora":
            T = _log(rng, 1, 2048)
            c = lora(T, _log(rng, 64, 28672), 256 * _log(rng, 1, 56), rng.choice(["f32", "f16", "bf16", "bf16"]),
                     rng.choice(["q8_0", "q4_0"]), rng.randint(1, 64), _log(rng, 1, 64), rng.randint(1, min(T, 64)),
                     rng.choice([0.0, 0.3]))
        elif op == "softmax":
            c = softmax(_log(rng, 1, 512), _log(rng, 100, 152000), rng.choice(["f32", "f16", "bf16"]), rng.randint(0, 1))
        else:
            c = verify(_log(rng, 1, 64), rng.randint(0, 8), _log(rng, 100, 152000), rng.randint(0, 1))
        if _cost(c) <= largest:
            return c


def _cost(c):
    w = work(c)
    times = 3 if c.get("dtype") == "f32" and c["op"] in ("moe", "lora") else 1
    return max(w["bytes"] / 6.8e12, times * w["flops"] / 1.9e15)


def work(case):
    c = case
    if c["op"] == "moe":
        E, k, T, e = c["n_experts"], c["n_active"], c["n_tokens"], 2 if c["dtype"] != "f32" else 4
        hit = E * (1 - (1 - k / E) ** T)                  # experts that some token picks, routing uniform
        xs = T * (k if c["per_slot"] else 1) * c["cols"] * e
        ys = {"none": T * k * c["rows"], "swiglu": T * k * c["rows"] // 2, "combine": T * c["rows"]}[c["epilogue"]] * e
        return {"bytes": hit * c["rows"] * c["cols"] // 32 * 34 + xs + ys + 4 * T * k,
                "flops": 2 * T * k * c["rows"] * c["cols"]}
    if c["op"] == "lora":
        T, e = c["n_tokens"], 2 if c["dtype"] != "f32" else 4
        used = min(c["n_adapters"], c["n_req"])
        return {"bytes": c["rows"] * c["cols"] // 32 * BLOCK_BYTES[c["fmt"]] + T * (c["cols"] + c["rows"]) * e
                + used * c["rank"] * (c["rows"] + c["cols"]) * 2,
                "flops": 2 * T * (c["rows"] * c["cols"] + c["rank"] * (c["rows"] + c["cols"]))}
    if c["op"] == "softmax":
        n = c["n_rows"] * c["vocab"]
        return {"bytes": n * (4 + (4 if c["dtype"] == "f32" else 2)), "flops": 4 * n}
    n = c["n_req"] * c["vocab"]
    return {"bytes": n * 4 * (1 if c["sure"] else 2) + 40 * c["n_req"], "flops": 3 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _blocks(g, fmt, rows, cols):
    """Weights of deviation 0.02 as stored blocks, [rows][cols / 32][34 or 18] bytes."""
    w = _normal(g, rows, cols // 32, 32, std=0.02)
    top = w.abs().amax(-1, keepdim=True)
    if fmt == "q8_0":
        d = (top / 127).half()
        q = (w / (top / 127).clamp_min(1e-30)).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        return torch.cat([d.view(torch.uint8), q], -1).contiguous()
    d = (top / -8).half()
    n = (w / d.float().clamp(max=-1e-30) + 8.5).floor().clamp(0, 15).to(torch.uint8)
    return torch.cat([d.view(torch.uint8), n[..., :16] | (n[..., 16:] << 4)], -1).contiguous()


def _exponents(blocks, fmt, n_mats):
    """One power of two a matrix, kept beside the weights: the largest |weight| a block scale allows is below 2^(e + 14)."""
    d = blocks[..., :2].contiguous().view(torch.float16).float().abs().reshape(n_mats, -1).amax(-1)
    return (torch.frexp(d * (128 if fmt == "q8_0" else 8))[1] - 14).to(torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c)}
    if c["op"] == "moe":
        E, k, T = c["n_experts"], c["n_active"], c["n_tokens"]
        s["W"] = torch.cat([_blocks(g, "q8_0", c["rows"], c["cols"]) for _ in range(E)])
        s["w_exp"] = _exponents(s["W"], "q8_0", E)
        popular = c["skew"] * _normal(g, 1, E) - torch.log(-torch.log(_uniform(g, T, E).clamp(1e-9, 1 - 1e-7)))
        s["ids"] = popular.topk(k, dim=1).indices.to(torch.int32).contiguous()
        x = _normal(g, T, k, c["cols"]) if c["per_slot"] else _normal(g, T, c["cols"])
        s["x"] = x.to(DTYPES[c["dtype"]])
        w = -torch.log(_uniform(g, T, k).clamp_min(1e-6))
        s["router_w"] = w / w.sum(1, keepdim=True)
    elif c["op"] == "lora":
        T, r = c["n_tokens"], c["rank"]
        s["W"] = _blocks(g, c["fmt"], c["rows"], c["cols"])
        s["w_exp"] = _exponents(s["W"], c["fmt"], 1)
        s["x"] = _normal(g, T, c["cols"]).to(DTYPES[c["dtype"]])
        s["A"] = _normal(g, c["n_adapters"], r, c["cols"], std=0.02).bfloat16()
        s["B"] = _normal(g, c["n_adapters"], c["rows"], r, std=0.02).bfloat16()
        s["scales"] = 0.25 + 2 * _uniform(g, c["n_adapters"])
        # each request's tokens follow one another; its length and its adapter are its own
        cuts = torch.randperm(T - 1, generator=g, device=DEV)[:c["n_req"] - 1] + 1 if T > 1 else torch.empty(0, device=DEV)
        req = torch.zeros(T, dtype=torch.int64, device=DEV)
        req[cuts.long()] = 1
        req = req.cumsum(0)
        adapter = torch.randint(0, c["n_adapters"], (T,), generator=g, device=DEV)
        adapter[_uniform(g, T) < c["bare"]] = -1
        s["ids"] = adapter[req].to(torch.int32)
    elif c["op"] == "softmax":
        l = _normal(g, c["n_rows"], c["vocab"], std=2.5)
        l[:, ::97] = -math.inf                              # tokens that a grammar rules out
        l[:, 0] = 0.5
        s["logits"] = l.to(DTYPES[c["dtype"]])
        t = 0.3 + _uniform(g, c["n_rows"])
        t[::5] = 0.0                                        # some requests are greedy
        s["t"] = t if c["warm"] else None
    else:
        R, V = c["n_req"], c["vocab"]
        # 0 to `most` drafts a request in mixed order; the lengths are the case's, what is drafted is the seed's
        n = torch.tensor([c["most"] if R == 1 else (((r + 1) * 2654435761 >> 12) & 0xFFFF) % (c["most"] + 1) for r in range(R)], device=DEV)
        off = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
        off[1:] = n.cumsum(0)
        D = int(off[-1])
        target = _normal(g, D + R, V, std=2.5)
        s["p"] = torch.softmax(target, -1)
        # the draft model's logits are the target's with an error of its own
        at = torch.arange(D, device=DEV) + torch.repeat_interleave(torch.arange(R, device=DEV), n)
        q = torch.softmax(target[at] + _normal(g, D, V, std=0.6), -1)
        s["drafts"] = (torch.multinomial(q, 1, generator=g)[:, 0] if D else torch.empty(0, device=DEV)).to(torch.int32)
        s["q"] = None if c["sure"] else q
        s["off"] = off
        s["u"], s["u_sample"] = _uniform(g, D), _uniform(g, R)
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import quantized_weight_matvec_hq_gb300 as hq
    c = s["case"]
    dt = c.get("dtype")
    if "y" not in s:                                        # outputs and workspace, made once as a program does
        if c["op"] == "moe":
            T, k = c["n_tokens"], c["n_active"]
            shape = {"none": (T, k, c["rows"]), "swiglu": (T, k, c["rows"] // 2), "combine": (T, c["rows"])}[c["epilogue"]]
            s["y"] = torch.empty(shape, dtype=DTYPES[dt], device=DEV)
            s["epi"] = {"none": hq.HQ_MOE_EPI_NONE, "swiglu": hq.HQ_MOE_EPI_SWIGLU, "combine": hq.HQ_MOE_EPI_COMBINE}[c["epilogue"]]
            n = hq.hq_moe_matmul_workspace(c["n_experts"], k, c["rows"], c["cols"], T, c["per_slot"], hq.DTYPE_CODES[dt], s["epi"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        elif c["op"] == "lora":
            s["y"] = torch.empty((c["n_tokens"], c["rows"]), dtype=DTYPES[dt], device=DEV)
            n = hq.hq_matmul_adapters_workspace(c["rank"], c["rows"], c["cols"], c["n_tokens"], hq.DTYPE_CODES[dt])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        elif c["op"] == "softmax":
            s["y"] = torch.empty((c["n_rows"], c["vocab"]), dtype=torch.float32, device=DEV)
        else:
            s["y"] = torch.empty(c["n_req"], dtype=torch.int32, device=DEV)
            s["tokens"] = torch.empty(s["p"].shape[0], dtype=torch.int32, device=DEV)
    if c["op"] == "moe":
        hq.hq_moe_matmul_q8_0(s["W"], s["w_exp"], s["ids"], s["x"], c["per_slot"],
                              s["router_w"] if c["epilogue"] == "combine" else None, s["y"], c["n_experts"], c["n_active"],
                              c["rows"], c["cols"], c["n_tokens"], hq.DTYPE_CODES[dt], s["epi"], s["ws"], s["ws"].numel())
        return s["y"]
    if c["op"] == "lora":
        fn = hq.hq_matmul_q8_0_adapters if c["fmt"] == "q8_0" else hq.hq_matmul_q4_0_adapters
        fn(s["W"], s["w_exp"], s["x"], s["ids"], s["A"], s["B"], s["scales"], c["n_adapters"], c["rank"], s["y"], c["rows"],
           c["cols"], c["n_tokens"], hq.DTYPE_CODES[dt], s["ws"], s["ws"].numel())
        return s["y"]
    if c["op"] == "softmax":
        hq.hq_softmax_rows(s["logits"], s["t"], s["y"], c["n_rows"], c["vocab"], hq.DTYPE_CODES[dt])
        return s["y"]
    hq.hq_verify_drafts(s["p"], s["q"], s["drafts"], s["off"], s["u"], s["u_sample"], s["y"], s["tokens"], c["n_req"],
                        s["drafts"].numel(), c["vocab"])
    return {"accepted": s["y"], "tokens": s["tokens"]}


def _weights(blocks, fmt, dtype=torch.float32):
    """[..., blocks, bytes] -> [..., cols] weights."""
    d = blocks[..., :2].contiguous().view(torch.float16).to(dtype)
    if fmt == "q8_0":
        q = blocks[..., 2:].view(torch.int8).to(dtype)
    else:
        b = blocks[..., 2:]
        q = torch.cat([b & 15, b >> 4], -1).to(dtype) - 8
    return (d * q).flatten(-2)


def _plain(s):
    c = s["case"]
    if c["op"] == "moe":
        T, k, rows, cols = c["n_tokens"], c["n_active"], c["rows"], c["cols"]
        used, which, count = torch.unique(s["ids"].flatten(), return_inverse=True, return_counts=True)
        w = _weights(s["W"].view(c["n_experts"], rows, cols // 32, 34)[used.long()], "q8_0")
        order = which.argsort()
        place = torch.empty_like(order)
        place[order] = torch.arange(T * k, device=DEV) - (count.cumsum(0) - count)[which[order]]
        x = s["x"].float()
        x = x.view(T * k, cols) if c["per_slot"] else x.repeat_interleave(k, 0)
        groups = torch.zeros(len(used), int(count.max()), cols, device=DEV)
        groups[which, place] = x
        y = torch.bmm(groups, w.transpose(1, 2))[which, place].view(T, k, rows)
        if c["epilogue"] == "swiglu":
            y = y[..., 0::2] / (1 + torch.exp(-y[..., 0::2])) * y[..., 1::2]
        elif c["epilogue"] == "combine":
            y = (y * s["router_w"][..., None]).sum(1)
        return y.to(DTYPES[c["dtype"]])
    if c["op"] == "lora":
        T, r, n = c["n_tokens"], c["rank"], c["n_adapters"]
        x = s["x"].float()
        y = x @ _weights(s["W"], c["fmt"]).T
        u = (x @ s["A"].float().view(n * r, -1).T).view(T, n, r)
        u = u * ((s["ids"][:, None] == torch.arange(n, device=DEV)) * s["scales"])[..., None]
        y = y + u.view(T, n * r) @ s["B"].float().transpose(1, 2).reshape(n * r, -1)
        return y.to(DTYPES[c["dtype"]])
    if c["op"] == "softmax":
        l = s["logits"].float()
        t = torch.ones(c["n_rows"], device=DEV) if s["t"] is None else s["t"]
        e = torch.exp((l - l.amax(-1, keepdim=True)) / t.clamp_min(1e-30)[:, None])
        p = e / e.sum(-1, keepdim=True)
        place = torch.arange(c["vocab"], device=DEV)
        greedy = place == torch.where(l == l.amax(-1, keepdim=True), place, c["vocab"]).amin(-1, keepdim=True)
        return torch.where((t > 0)[:, None], p, greedy.float())
    R, V, D = c["n_req"], c["vocab"], s["drafts"].numel()
    off = s["off"].long()
    n = off[1:] - off[:-1]
    req = torch.repeat_interleave(torch.arange(R, device=DEV), n, output_size=D)
    at = torch.arange(D, device=DEV)
    tok = s["drafts"].long()
    ok = s["u"] * (torch.ones_like(s["u"]) if s["q"] is None else s["q"][at, tok]) < s["p"][at + req, tok]
    bad = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), (~ok).long().cumsum(0)])   # refused drafts before each
    good = (bad[1:] == bad[off[:-1]][req]).long()
    acc = torch.zeros(R, dtype=torch.int64, device=DEV).index_add_(0, req, good)
    r = s["p"][off[:-1] + torch.arange(R, device=DEV) + acc]
    rest = (acc < n)[:, None]
    if D:
        i = (off[:-1] + acc).clamp_max(D - 1)
        q = torch.arange(V, device=DEV) == tok[i][:, None] if s["q"] is None else s["q"][i]
        left = torch.where(rest, (r - q.float()).clamp_min(0), r)
    else:
        left = r
    steps = torch.floor(left * 2.0 ** 40).long()
    steps = torch.where(steps.sum(-1, keepdim=True) > 0, steps, torch.floor(r * 2.0 ** 40).long())
    c_ = steps.cumsum(-1)
    u = torch.floor(s["u_sample"] * 2.0 ** 24).long()
    goal = (c_[:, -1] >> 24) * u + (((c_[:, -1] & 0xFFFFFF) * u) >> 24)
    pick = (c_ <= goal[:, None]).sum(-1)
    row = torch.arange(D + R, device=DEV)
    of = torch.repeat_interleave(torch.arange(R, device=DEV), n + 1, output_size=D + R)
    i = row - (off[:-1] + torch.arange(R, device=DEV))[of]
    drafted = tok[(row - of).clamp(0, max(D - 1, 0))] if D else torch.zeros_like(row)
    tokens = torch.where(i < acc[of], drafted, torch.where(i == acc[of], pick[of], -1))
    return {"accepted": acc.to(torch.int32), "tokens": tokens.to(torch.int32)}


# ------------------------------------------------------------------ the same in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "moe":
        T, k, rows, cols = c["n_tokens"], c["n_active"], c["rows"], c["cols"]
        x = s["x"].to(f64).reshape(T, -1, cols)
        y = torch.zeros(T, k, rows, dtype=f64, device=DEV)
        bank = s["W"].view(c["n_experts"], rows, cols // 32, 34)
        for e in range(c["n_experts"]):
            t, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
            if len(t):
                b = bank[e]
                w = b[:, :, :2].contiguous().view(torch.float16).to(f64) * b[:, :, 2:].contiguous().view(torch.int8).to(f64)
                y[t, slot] = x[t, slot if c["per_slot"] else 0] @ w.reshape(rows, cols).T
        if c["epilogue"] == "swiglu":
            gate, up = y.unflatten(-1, (rows // 2, 2)).unbind(-1)
            return gate * torch.sigmoid(gate) * up
        return torch.einsum("tkr,tk->tr", y, s["router_w"].to(f64)) if c["epilogue"] == "combine" else y
    if c["op"] == "lora":
        b = s["W"]
        d = b[:, :, :2].contiguous().view(torch.float16).to(f64)
        if c["fmt"] == "q8_0":
            q = b[:, :, 2:].contiguous().view(torch.int8).to(f64)
        else:
            q = torch.stack([b[:, :, 2:].remainder(16), b[:, :, 2:].div(16, rounding_mode="floor")], 2).flatten(2).to(f64) - 8
        x = s["x"].to(f64)
        y = x @ (d * q).reshape(c["rows"], c["cols"]).T
        for a in range(c["n_adapters"]):
            t = torch.nonzero(s["ids"] == a)[:, 0]
            if len(t):
                y[t] += s["scales"][a].to(f64) * ((x[t] @ s["A"][a].to(f64).T) @ s["B"][a].to(f64).T)
        return y
    if c["op"] == "softmax":
        l = s["logits"].to(f64)
        p = torch.empty_like(l)
        for i in range(c["n_rows"]):
            t = 1.0 if s["t"] is None else float(s["t"][i])
            if t > 0:
                p[i] = torch.softmax(l[i] / t, -1)
            else:
                p[i] = 0.0
                p[i, int(torch.nonzero(l[i] == l[i].max())[0])] = 1.0
        return p
    off, drafts, u, us = (s[k].cpu().tolist() for k in ("off", "drafts", "u", "u_sample"))
    accepted, tokens = [], []
    for r in range(c["n_req"]):
        n, a = off[r + 1] - off[r], 0
        while a < n:
            i, d = off[r] + a, drafts[off[r] + a]
            q = 1.0 if s["q"] is None else float(s["q"][i, d])
            if not float(torch.tensor(u[i], dtype=torch.float32) * torch.tensor(q, dtype=torch.float32)) < float(s["p"][i + r, d]):
                break
            a += 1
        p = s["p"][off[r] + r + a]
        left = p
        if a < n:
            q = torch.zeros_like(p) if s["q"] is None else s["q"][off[r] + a]
            if s["q"] is None:
                q[drafts[off[r] + a]] = 1.0
            left = (p - q).clamp_min(0)
        steps = (left.to(f64) * 2.0 ** 40).floor().to(torch.int64)
        if int(steps.sum()) == 0:
            steps = (p.to(f64) * 2.0 ** 40).floor().to(torch.int64)
        goal = int(steps.sum()) * int(us[r] * 2 ** 24) // 2 ** 24
        accepted.append(a)
        tokens += drafts[off[r]:off[r] + a] + [int(torch.searchsorted(steps.cumsum(0), goal, right=True))] + [-1] * (n - a)
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "tokens": torch.tensor(tokens, dtype=torch.int32)}
