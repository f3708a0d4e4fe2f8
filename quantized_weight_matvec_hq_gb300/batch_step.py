"""One step of a batch server, over the many-token calls of the library.

Several requests are verified together: request r brings the tokens it drafted
and the token before them, n_r + 1 positions.  All positions go through

  1. hq_moe_matmul_q8_0, SwiGLU epilogue      a feed-forward layer's gate|up product, each position at its experts
  2. hq_moe_matmul_q8_0, combine epilogue     its down product and the router-weighted sum
  3. hq_matmul_q8_0_adapters                  the vocabulary projection, each position with its request's adapter
  4. hq_softmax_rows                          probabilities at each request's temperature
  5. hq_verify_drafts                         accepted drafts, and one sampled token a request

With an `Attention`, an attention layer over a quantized key/value cache comes before them:

  a. hq_matmul_q8_0_adapters (no adapters)    queries, keys and values of all positions, side by side
  b. hq_cache_write                           keys and values into the cache
  c. hq_cache_attention                       each position over its request's cached ones
  d. hq_matmul_q8_0_adapters (no adapters)    the output projection, whose rows steps 1 to 5 then take for x

The positions of rejected drafts need no clean-up: the next step's lengths put its tokens over them.

    step = BatchStep(gate_up, down, head, (lora_A, lora_B, scales), n_experts=128, n_active=8, hidden=2048, ffn=768,
                     vocab=151936, most_tokens=512, dtype="bf16")
    n_accepted, tokens = step(x, expert_ids, router_w, adapter_ids, temperature, drafts, offsets, u_accept, u_sample)

The calls run on one stream without a host synchronisation and allocate nothing
but the tensors that this class keeps, so a step with fixed sizes can be
captured in a CUDA graph.

    python -m quantized_weight_matvec_hq_gb300.batch_step      # a small model with random weights
"""
from __future__ import annotations

import numpy as np
import torch

import quantized_weight_matvec_hq_gb300 as hq

TORCH_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DTYPE_OF = {t: hq.DTYPE_CODES[name] for name, t in TORCH_DTYPES.items()}


def positions(offsets) -> tuple[np.ndarray, np.ndarray]:
    """Of every position, in order, its request and its number in the request: request r has
    offsets[r + 1] - offsets[r] + 1 of them, the first at offsets[r] + r."""
    n = np.diff(np.asarray(offsets, np.int64)) + 1
    request = np.repeat(np.arange(len(n)), n)
    return request, np.arange(len(request)) - (np.asarray(offsets, np.int64)[request] + request)


def position_offsets(offsets):
    """Of draft offsets, those of the positions: request r's begin at offsets[r] + r."""
    return offsets + torch.arange(offsets.shape[0], dtype=offsets.dtype, device=offsets.device)


def _expect(name, t, shape, dtype, device=None):
    """The library's calls take addresses: what a tensor holds is checked here."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name}: {tuple(shape)} of {dtype}, contiguous{'' if device is None else f' on {device}'}, expected; "
                         f"got {tuple(t.shape)} of {t.dtype}, strides {t.stride()}, on {t.device}")


def _expect_current(device):
    """The library's calls run on the current device, whatever device their addresses are of."""
    if device.type != "cuda" or device.index != torch.cuda.current_device():
        raise ValueError(f"calls run on the current CUDA device; what they were given is on {device}")


class KeyValueCache:
    """A paged key/value cache in blocks of Q8_0 or Q4_0, and the library's calls on it.  A batch is told of by
    (offsets, lengths, page_table), int32 device tensors as hq_cache_write takes them; the pages are the caller's to hand out.
    Calls with another device current than the cache's are refused with a ValueError."""

    def __init__(self, fmt, n_pages, page_size, n_kv_heads, head_dim, device="cuda"):
        self.fmt, self.n_pages, self.page, self.kv, self.dim = hq.FMT_CODES[fmt], n_pages, page_size, n_kv_heads, head_dim
        self.pool = torch.empty(n_pages * hq.hq_cache_page_bytes(self.fmt, n_kv_heads, head_dim, page_size), dtype=torch.uint8,
                                device=device)
        self.device = self.pool.device

    def _batch(self, batch, T):
        offsets, lengths, table = batch
        R = lengths.shape[0]
        _expect("offsets", offsets, (R + 1,), torch.int32, self.device)
        _expect("lengths", lengths, (R,), torch.int32, self.device)
        _expect("page_table", table, (R, table.shape[-1]), torch.int32, self.device)
        return self.pool, self.n_pages, self.page, table, table.shape[-1], offsets, lengths, R, T

    def _rows(self, name, t, heads, dtype=None):
        """[tokens][heads][head_dim], a token's heads together: of any stride from token to token."""
        if t.ndim != 3 or t.shape[1:] != (heads, self.dim) or t.device != self.device or t.dtype != (dtype or t.dtype) or \
                t.dtype not in TORCH_DTYPES.values() or (t.shape[0] > 0 and (t.stride(2) != 1 or t.stride(1) != self.dim)):
            raise ValueError(f"{name}: [tokens][{heads}][{self.dim}], a token's heads together, on {self.device} expected; got "
                             f"{tuple(t.shape)} of {t.dtype}, strides {t.stride()}, on {t.device}")
        return t, heads * self.dim if t.shape[0] < 2 else t.stride(0)          # (one token's may be anything)

    def write(self, k, v, batch, stream=None):
        """k and v [tokens][n_kv_heads][head_dim] to their positions (hq_cache_write)."""
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"{k.shape[0]} tokens of keys, {v.shape[0]} of values")
        args = *self._rows("k", k, self.kv), *self._rows("v", v, self.kv, k.dtype), *self._batch(batch, k.shape[0])
        _expect_current(self.device)
        hq.hq_cache_write(self.fmt, *args, self.kv, self.dim, DTYPE_OF[k.dtype], stream=stream)

    def read(self, k, v, batch, stream=None):
        """The values of the tokens' positions into k and v (hq_cache_read)."""
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"{k.shape[0]} tokens of keys, {v.shape[0]} of values")
        args = *self._rows("k", k, self.kv), *self._rows("v", v, self.kv, k.dtype), *self._batch(batch, k.shape[0])
        _expect_current(self.device)
        hq.hq_cache_read(self.fmt, *args, self.kv, self.dim, DTYPE_OF[k.dtype], stream=stream)

    def workspace_bytes(self, n_req, table_width, n_tokens, n_heads, dtype):
        """Of a batch, and of every one of fewer tokens or requests (hq_cache_attention_workspace)."""
        return hq.hq_cache_attention_workspace(self.fmt, self.page, table_width, n_req, n_tokens, n_heads, self.kv, self.dim,
                                               hq.DTYPE_CODES[dtype])

    def attend(self, q, out, batch, workspace, scale=None, causal=True, window=0, stream=None):
        """q [tokens][heads][head_dim] over the cache, into out (hq_cache_attention); scale: 1 / sqrt(head_dim) if None."""
        heads = q.shape[1]
        if out.shape != q.shape:
            raise ValueError(f"out: {tuple(q.shape)} expected; got {tuple(out.shape)}")
        args = self._batch(batch, q.shape[0])
        q, q_stride = self._rows("q", q, heads)
        out, out_stride = self._rows("out", out, heads, q.dtype)
        _expect("workspace", workspace, (workspace.numel(),), torch.uint8, self.device)
        _expect_current(self.device)
        hq.hq_cache_attention(self.fmt, q, q_stride, *args, heads, self.kv, self.dim, self.dim ** -0.5 if scale is None else scale,
                              int(causal), window, out, out_stride, DTYPE_OF[q.dtype], workspace, workspace.numel(), stream=stream)


class Attention:
    """The attention layer of a step: qkv: Q8_0 blocks of [(n_heads + 2 n_kv_heads) head_dim][hidden], out: of
    [hidden][n_heads head_dim] (uint8 device tensors), over a KeyValueCache; a request has at most
    `most_pages` pages.  window: 0, or how many positions a token looks back on, its own included.  There are no norms, rotary
    positions or residual sums in it: a model with those calls KeyValueCache between its own steps."""

    def __init__(self, qkv, out, n_heads, cache, most_pages, window=0):
        self.qkv, self.out, self.heads, self.cache, self.most_pages, self.window = qkv, out, n_heads, cache, most_pages, window


class BatchStep:
    def __init__(self, gate_up, down, head, adapters, *, n_experts, n_active, hidden, ffn, vocab, most_tokens, dtype="bf16",
                 attention=None):
        """gate_up: Q8_0 blocks of [n_experts][2 ffn][hidden] (gate and up rows interleaved), down: of
        [n_experts][hidden][ffn], head: of [vocab][hidden]; uint8 device tensors.  adapters: (A, B, scales) as
        hq_matmul_q8_0_adapters takes them, or None.  attention: an Attention, or None.  Steps may run on another stream than the current one if it comes
        behind it (the set-up of the weights runs here)."""
        dev = gate_up.device
        for name, W, rows, cols in (("gate_up", gate_up, n_experts * 2 * ffn, hidden), ("down", down, n_experts * hidden, ffn),
                                    ("head", head, vocab, hidden)):
            _expect(name, W.view(-1) if W.is_contiguous() else W, (rows * (cols // hq.QK) * hq.Q8_0_BLOCK_BYTES,), torch.uint8, dev)
        if adapters is not None:
            n, rank = adapters[0].shape[:2]
            _expect("lora_A", adapters[0], (n, rank, hidden), torch.bfloat16, dev)
            _expect("lora_B", adapters[1], (n, vocab, rank), torch.bfloat16, dev)
            _expect("scales", adapters[2], (n,), torch.float32, dev)
        self.gate_up, self.down, self.head = gate_up, down, head
        self.A, self.B, self.scales = adapters if adapters is not None else (None, None, None)
        self.n_adapters, self.rank = (self.A.shape[0], self.A.shape[1]) if adapters is not None else (0, 1)
        self.E, self.k, self.hidden, self.ffn, self.vocab, self.most = n_experts, n_active, hidden, ffn, vocab, most_tokens
        self.dtype_name = dtype
        self.dtype, self.x_dtype, self.device = hq.DTYPE_CODES[dtype], TORCH_DTYPES[dtype], dev
        _expect_current(dev)

        def exponents(W, mats, rows, cols):
            e = torch.empty(mats, dtype=torch.int32, device=dev)
            hq.hq_weight_exponents(hq.FMT_CODES["q8_0"], W, e, mats, rows, cols)
            return e
        self.e_gate_up = exponents(gate_up, n_experts, 2 * ffn, hidden)
        self.e_down = exponents(down, n_experts, hidden, ffn)
        self.e_head = exponents(head, 1, vocab, hidden)
        t = TORCH_DTYPES[dtype]
        self.attention = attention
        if attention is not None:
            c, H, D = attention.cache, attention.heads, attention.cache.dim
            self.width = (H + 2 * c.kv) * D
            for name, W, rows, cols in (("qkv", attention.qkv, self.width, hidden), ("out", attention.out, hidden, H * D)):
                _expect(name, W, (rows * (cols // hq.QK) * hq.Q8_0_BLOCK_BYTES,), torch.uint8, dev)
            self.e_qkv = exponents(attention.qkv, 1, self.width, hidden)
            self.e_out = exponents(attention.out, 1, hidden, H * D)
            self.rows = torch.empty((most_tokens, H + 2 * c.kv, D), dtype=t, device=dev)
            self.seen = torch.empty((most_tokens, H, D), dtype=t, device=dev)
            self.x = torch.empty((most_tokens, hidden), dtype=t, device=dev)
        self.workspace = torch.empty(self._workspace_bytes(most_tokens), dtype=torch.uint8, device=dev)
        self.h = torch.empty((most_tokens, n_active, ffn), dtype=t, device=dev)
        self.y = torch.empty((most_tokens, hidden), dtype=t, device=dev)
        self.logits = torch.empty((most_tokens, vocab), dtype=t, device=dev)
        self.p = torch.empty((most_tokens, vocab), dtype=torch.float32, device=dev)
        self.n_accepted = torch.empty(most_tokens, dtype=torch.int32, device=dev)
        self.tokens = torch.empty(most_tokens, dtype=torch.int32, device=dev)

    def _workspace_bytes(self, T):
        need = (hq.hq_moe_matmul_workspace(self.E, self.k, 2 * self.ffn, self.hidden, T, 0, self.dtype, hq.HQ_MOE_EPI_SWIGLU),
                hq.hq_moe_matmul_workspace(self.E, self.k, self.hidden, self.ffn, T, 1, self.dtype, hq.HQ_MOE_EPI_COMBINE),
                hq.hq_matmul_adapters_workspace(self.rank, self.vocab, self.hidden, T, self.dtype))
        if self.attention is not None:
            a, c = self.attention, self.attention.cache
            need += (hq.hq_matmul_adapters_workspace(1, self.width, self.hidden, T, self.dtype),
                     hq.hq_matmul_adapters_workspace(1, self.hidden, a.heads * c.dim, T, self.dtype),
                     c.workspace_bytes(T, a.most_pages, T, a.heads, self.dtype_name))
        if min(need) < 0:
            raise ValueError("sizes that the library refuses")
        return max(1, *need)

    def _attend(self, x, cache, T, R, stream):
        a, c, ws = self.attention, self.attention.cache, self.workspace
        offsets, lengths, table = cache
        if lengths.shape[0] != R or table.shape[-1] > a.most_pages:
            raise ValueError(f"a cache of {lengths.shape[0]} requests and {table.shape[-1]} pages each, for {R} requests, {a.most_pages} pages at most")
        _expect("x", x, (T, self.hidden), self.x_dtype, self.device)
        hq.hq_matmul_q8_0_adapters(a.qkv, self.e_qkv, x, None, None, None, None, 0, 1, self.rows, self.width, self.hidden, T,
                                   self.dtype, ws, ws.numel(), stream=stream)
        rows = self.rows[:T]
        c.write(rows[:, a.heads:a.heads + c.kv], rows[:, a.heads + c.kv:], cache, stream=stream)
        c.attend(rows[:, :a.heads], self.seen[:T], cache, ws, window=a.window, stream=stream)
        hq.hq_matmul_q8_0_adapters(a.out, self.e_out, self.seen, None, None, None, None, 0, 1, self.x, self.hidden,
                                   a.heads * c.dim, T, self.dtype, ws, ws.numel(), stream=stream)
        return self.x[:T]

    def _check_inputs(self, x, expert_ids, router_w, adapter_ids, temperature, drafts, offsets, u_accept, u_sample, q):
        T, D, R = x.shape[0], drafts.shape[0], u_sample.shape[0]
        i32, f32 = torch.int32, torch.float32
        for name, t, shape, dtype in (("x", x, (T, self.hidden), self.x_dtype), ("expert_ids", expert_ids, (T, self.k), i32),
                                      ("router_w", router_w, (T, self.k), f32), ("drafts", drafts, (D,), i32),
                                      ("offsets", offsets, (R + 1,), i32), ("u_accept", u_accept, (D,), f32),
                                      ("u_sample", u_sample, (R,), f32)):
            _expect(name, t, shape, dtype, self.device)
        if self.n_adapters:
            _expect("adapter_ids", adapter_ids, (T,), i32, self.device)
        if temperature is not None:
            _expect("temperature", temperature, (T,), f32, self.device)
        if q is not None:
            _expect("q", q, (D, self.vocab), f32, self.device)

    def __call__(self, x, expert_ids, router_w, adapter_ids, temperature, drafts, offsets, u_accept, u_sample, q=None,
                 cache=None, stream=None):
        """x [T][hidden], expert_ids int32 and router_w fp32 [T][n_active], adapter_ids int32 and temperature fp32 [T],
        for the T = len(drafts) + len(u_sample) positions; the rest as hq_verify_drafts takes it, device
        tensors all, on the current device; others are refused with a ValueError.  cache (with an Attention): (position_offsets(offsets), lengths,
        page_table), lengths with this step's positions in them.  Returns its n_accepted and tokens, which the next call overwrites."""
        T, R = x.shape[0], u_sample.shape[0]
        if T != drafts.shape[0] + R or T > self.most:
            raise ValueError(f"{T} positions for {drafts.shape[0]} drafts and {R} requests, {self.most} at most")
        self._check_inputs(x, expert_ids, router_w, adapter_ids, temperature, drafts, offsets, u_accept, u_sample, q)
        if (cache is not None) != (self.attention is not None):
            raise ValueError("a cache is given with an Attention, and only then")
        _expect_current(self.device)
        ws = self.workspace
        if self.attention is not None:
            x = self._attend(x, cache, T, R, stream)
        hq.hq_moe_matmul_q8_0(self.gate_up, self.e_gate_up, expert_ids, x, 0, None, self.h, self.E, self.k, 2 * self.ffn,
                              self.hidden, T, self.dtype, hq.HQ_MOE_EPI_SWIGLU, ws, ws.numel(), stream=stream)
        hq.hq_moe_matmul_q8_0(self.down, self.e_down, expert_ids, self.h, 1, router_w, self.y, self.E, self.k, self.hidden,
                              self.ffn, T, self.dtype, hq.HQ_MOE_EPI_COMBINE, ws, ws.numel(), stream=stream)
        hq.hq_matmul_q8_0_adapters(self.head, self.e_head, self.y, adapter_ids, self.A, self.B, self.scales, self.n_adapters,
                                   self.rank, self.logits, self.vocab, self.hidden, T, self.dtype, ws, ws.numel(),
                                   stream=stream)
        hq.hq_softmax_rows(self.logits, temperature, self.p, T, self.vocab, self.dtype, stream=stream)
        hq.hq_verify_drafts(self.p, q, drafts, offsets, u_accept, u_sample, self.n_accepted, self.tokens, R,
                            drafts.shape[0], self.vocab, stream=stream)
        return self.n_accepted[:R], self.tokens[:T]


def random_inputs(g, drafted, *, n_experts, n_active, hidden, vocab, n_adapters, dtype="bf16", device="cuda"):
    """Inputs of a step for requests that drafted `drafted[r]` tokens each."""
    from quantized_weight_matvec_hq_gb300 import synthetic

    def put(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)
    offsets = np.concatenate([[0], np.cumsum(drafted)]).astype(np.int32)
    request, _ = positions(offsets)
    T, R, D = len(request), len(drafted), int(offsets[-1])
    adapter_of = g.integers(-1, n_adapters, R)
    temperature_of = np.where(g.uniform(0, 1, R) < 0.25, 0.0, g.uniform(0.5, 1.5, R))
    return dict(x=put(g.standard_normal((T, hidden)).astype(np.float32)).to(TORCH_DTYPES[dtype]),
                expert_ids=put(synthetic.expert_ids(g, T, n_active, n_experts)),
                router_w=put(synthetic.router_weights(g, T, n_active)),
                adapter_ids=put(adapter_of[request].astype(np.int32)),
                temperature=put(temperature_of[request].astype(np.float32)),
                drafts=put(g.integers(0, vocab, D).astype(np.int32)), offsets=put(offsets),
                u_accept=put(g.uniform(0, 1, D).astype(np.float32)), u_sample=put(g.uniform(0, 1, R).astype(np.float32)))


def random_step(g, *, n_experts, n_active, hidden, ffn, vocab, n_adapters, rank, most_tokens, dtype="bf16", device="cuda",
                n_heads=0, cache=None, most_pages=1, window=0):
    """A step over random weights, quantized on the device; with a KeyValueCache, an attention layer of n_heads over it."""
    def blocks(rows, cols):
        W = torch.from_numpy((g.standard_normal((rows, cols)) * 0.05).astype(np.float32)).to(device)
        out = torch.empty(rows * (cols // 32) * 34, dtype=torch.uint8, device=device)
        hq.hq_quantize_q8_0(W, out, rows, cols)
        return out

    def bf16(*shape):
        return torch.from_numpy((g.standard_normal(shape) * 0.05).astype(np.float32)).bfloat16().to(device)
    adapters = (bf16(n_adapters, rank, hidden), bf16(n_adapters, vocab, rank),
                torch.from_numpy(g.uniform(0.5, 2, n_adapters).astype(np.float32)).to(device))
    weights = blocks(n_experts * 2 * ffn, hidden), blocks(n_experts * hidden, ffn), blocks(vocab, hidden)
    attention = None
    if cache is not None:
        attention = Attention(blocks((n_heads + 2 * cache.kv) * cache.dim, hidden), blocks(hidden, n_heads * cache.dim), n_heads,
                              cache, most_pages, window)
    return BatchStep(*weights, adapters, n_experts=n_experts, n_active=n_active, hidden=hidden, ffn=ffn, vocab=vocab,
                     most_tokens=most_tokens, dtype=dtype, attention=attention)


def random_cache(g, cache, lengths, most_pages):
    """Pages for requests of these lengths, in mixed order, and what a step is told: (lengths, page_table)."""
    need = -(-np.asarray(lengths) // cache.page)
    if need.sum() > cache.n_pages or need.max(initial=0) > most_pages:
        raise ValueError(f"{need.sum()} pages needed, {cache.n_pages} there; {most_pages} a request at most")
    table = np.zeros((len(lengths), most_pages), np.int32)
    order, at = g.permutation(cache.n_pages), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return (torch.from_numpy(np.asarray(lengths, np.int32)).to(cache.device), torch.from_numpy(table).to(cache.device))


def main() -> None:
    from quantized_weight_matvec_hq_gb300 import synthetic
    g = synthetic.rng(synthetic.SEED_BASE)
    size = dict(n_experts=16, n_active=4, hidden=1024, vocab=8192, n_adapters=3)
    drafted = [4, 0, 7, 2, 1]
    cache = KeyValueCache("q4_0", n_pages=64, page_size=32, n_kv_heads=2, head_dim=128)
    step = random_step(g, ffn=512, rank=16, most_tokens=32, n_heads=8, cache=cache, most_pages=16, **size)
    cached = [40, 3, 300, 129, 0]                 # positions before this step, here of random rows
    lengths, table = random_cache(g, cache, [n + d + 1 for n, d in zip(cached, drafted)], 16)
    ends = np.concatenate([[0], np.cumsum(lengths.cpu().numpy())]).astype(np.int32)
    k, v = (torch.from_numpy(g.standard_normal((int(ends[-1]), 2, 128)).astype(np.float32)).cuda() for _ in "kv")
    cache.write(k, v, (torch.from_numpy(ends).cuda(), lengths, table))
    inputs = random_inputs(g, drafted, **size)
    n_accepted, tokens = step(**inputs, cache=(position_offsets(inputs["offsets"]), lengths, table))
    torch.cuda.synchronize()
    fault = hq.hq_device_fault()
    first = 0
    for r, n in enumerate(drafted):
        print(f"request {r}: drafted {n}, accepted {int(n_accepted[r])}, tokens {tokens[first:first + n + 1].tolist()}")
        first += n + 1
    if fault:
        raise SystemExit(f"device fault {fault:#x}")


if __name__ == "__main__":
    main()
