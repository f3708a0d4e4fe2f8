"""One step of a batch server, over the many-token calls of the library.

Several requests are verified together: request r brings the tokens it drafted
and the token before them, n_r + 1 positions.  All positions go through

  1. hq_moe_matmul_q8_0, SwiGLU epilogue      a feed-forward layer's gate|up product, each position at its experts
  2. hq_moe_matmul_q8_0, combine epilogue     its down product and the router-weighted sum
  3. hq_matmul_q8_0_adapters                  the vocabulary projection, each position with its request's adapter
  4. hq_softmax_rows                          probabilities at each request's temperature
  5. hq_verify_drafts                         accepted drafts, and one sampled token a request

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


def positions(offsets) -> tuple[np.ndarray, np.ndarray]:
    """Of every position, in order, its request and its number in the request: request r has
    offsets[r + 1] - offsets[r] + 1 of them, the first at offsets[r] + r."""
    n = np.diff(np.asarray(offsets, np.int64)) + 1
    request = np.repeat(np.arange(len(n)), n)
    return request, np.arange(len(request)) - (np.asarray(offsets, np.int64)[request] + request)


def _expect(name, t, shape, dtype, device=None):
    """The library's calls take addresses: what a tensor holds is checked here."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or (device is not None and t.device != device):
        raise ValueError(f"{name}: {tuple(shape)} of {dtype}, contiguous{'' if device is None else f' on {device}'}, expected; "
                         f"got {tuple(t.shape)} of {t.dtype}, strides {t.stride()}, on {t.device}")


class BatchStep:
    def __init__(self, gate_up, down, head, adapters, *, n_experts, n_active, hidden, ffn, vocab, most_tokens, dtype="bf16"):
        """gate_up: Q8_0 blocks of [n_experts][2 ffn][hidden] (gate and up rows interleaved), down: of
        [n_experts][hidden][ffn], head: of [vocab][hidden]; uint8 device tensors.  adapters: (A, B, scales) as
        hq_matmul_q8_0_adapters takes them, or None.  Steps may run on another stream than the current one if it comes
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
        self.dtype, self.x_dtype, self.device = hq.DTYPE_CODES[dtype], TORCH_DTYPES[dtype], dev

        def exponents(W, mats, rows, cols):
            e = torch.empty(mats, dtype=torch.int32, device=dev)
            hq.hq_weight_exponents(hq.FMT_CODES["q8_0"], W, e, mats, rows, cols)
            return e
        self.e_gate_up = exponents(gate_up, n_experts, 2 * ffn, hidden)
        self.e_down = exponents(down, n_experts, hidden, ffn)
        self.e_head = exponents(head, 1, vocab, hidden)
        self.workspace = torch.empty(self._workspace_bytes(most_tokens), dtype=torch.uint8, device=dev)
        t = TORCH_DTYPES[dtype]
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
        if min(need) < 0:
            raise ValueError("sizes that the library refuses")
        return max(1, *need)

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
                 stream=None):
        """x [T][hidden], expert_ids int32 and router_w fp32 [T][n_active], adapter_ids int32 and temperature fp32 [T],
        for the T = len(drafts) + len(u_sample) positions; the rest as hq_verify_drafts takes it, device
        tensors all; others are refused with a ValueError.  Returns its n_accepted and tokens, which the next call overwrites."""
        T, R = x.shape[0], u_sample.shape[0]
        if T != drafts.shape[0] + R or T > self.most:
            raise ValueError(f"{T} positions for {drafts.shape[0]} drafts and {R} requests, {self.most} at most")
        self._check_inputs(x, expert_ids, router_w, adapter_ids, temperature, drafts, offsets, u_accept, u_sample, q)
        ws = self.workspace
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


def random_step(g, *, n_experts, n_active, hidden, ffn, vocab, n_adapters, rank, most_tokens, dtype="bf16", device="cuda"):
    """A step over random weights, quantized on the device."""
    def blocks(rows, cols):
        W = torch.from_numpy((g.standard_normal((rows, cols)) * 0.05).astype(np.float32)).to(device)
        out = torch.empty(rows * (cols // 32) * 34, dtype=torch.uint8, device=device)
        hq.hq_quantize_q8_0(W, out, rows, cols)
        return out

    def bf16(*shape):
        return torch.from_numpy((g.standard_normal(shape) * 0.05).astype(np.float32)).bfloat16().to(device)
    adapters = (bf16(n_adapters, rank, hidden), bf16(n_adapters, vocab, rank),
                torch.from_numpy(g.uniform(0.5, 2, n_adapters).astype(np.float32)).to(device))
    return BatchStep(blocks(n_experts * 2 * ffn, hidden), blocks(n_experts * hidden, ffn), blocks(vocab, hidden), adapters,
                     n_experts=n_experts, n_active=n_active, hidden=hidden, ffn=ffn, vocab=vocab, most_tokens=most_tokens,
                     dtype=dtype)


def main() -> None:
    from quantized_weight_matvec_hq_gb300 import synthetic
    g = synthetic.rng(synthetic.SEED_BASE)
    size = dict(n_experts=16, n_active=4, hidden=1024, vocab=8192, n_adapters=3)
    drafted = [4, 0, 7, 2, 1]
    step = random_step(g, ffn=512, rank=16, most_tokens=32, **size)
    n_accepted, tokens = step(**random_inputs(g, drafted, **size))
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
