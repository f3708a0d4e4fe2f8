"""GPU tests of a step with an attention layer over a quantized cache: each stage against the 64-bit form of its own inputs,
steps that follow one another, and a captured step."""
from __future__ import annotations

import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import synthetic
from test_gpu_batch import U_OUT, assert_near, base_tol, dense, hq, no_device_fault  # noqa: F401
from test_gpu_cache import check_attention, stored, values

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SIZE = dict(n_experts=8, n_active=2, hidden=512, vocab=1000, n_adapters=3)


def make(g, dtype, fmt, heads, kv, dim, page, most_pages, most_tokens, window=0):
    from quantized_weight_matvec_hq_gb300 import batch_step
    cache = batch_step.KeyValueCache(fmt, 60, page, kv, dim)
    step = batch_step.random_step(g, ffn=256, rank=8, most_tokens=most_tokens, dtype=dtype, n_heads=heads, cache=cache,
                                  most_pages=most_pages, window=window, **SIZE)
    return cache, step


def fill(g, cache, lengths, table):
    """Random rows for every position; returns what is stored, by request, [length][kv][dim] keys and values."""
    ends = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    k, v = (g.standard_normal((int(ends[-1]), cache.kv, cache.dim)).astype(np.float32) for _ in "kv")
    cache.write(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                (torch.from_numpy(ends).cuda(), torch.from_numpy(np.asarray(lengths, np.int32)).cuda(), table))
    return [[x[a:b] for x in (k, v)] for a, b in zip(ends[:-1], ends[1:])]


@pytest.mark.parametrize("dtype,fmt,heads,kv,dim,window", [("bf16", "q4_0", 8, 2, 128, 0), ("f16", "q8_0", 4, 1, 64, 40),
                                                           ("f32", "q8_0", 6, 2, 128, 0), ("bf16", "q8_0", 24, 1, 256, 0)])
def test_steps_with_a_cache(hq, dtype, fmt, heads, kv, dim, window):
    """Two steps: the second's requests are longer by what the first accepted."""
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(1800 + dim)
    drafted, cached, page, W = [3, 0, 6, 1], [70, 5, 0, 200], 32, 10
    cache, step = make(g, dtype, fmt, heads, kv, dim, page, W, 40, window)
    total = [n + 16 for n in cached]
    _, table = batch_step.random_cache(g, cache, total, W)
    rows = fill(g, cache, total, table)
    here = np.asarray(cached)
    Wqkv = dense("q8_0", step.attention.qkv.cpu().numpy(), step.width, SIZE["hidden"])
    Wout = dense("q8_0", step.attention.out.cpu().numpy(), SIZE["hidden"], heads * dim)
    for _ in range(2):
        a = batch_step.random_inputs(g, drafted, dtype=dtype, **SIZE)
        new = np.asarray(drafted) + 1
        lengths = torch.from_numpy((here + new).astype(np.int32)).cuda()
        n_accepted, tokens = step(**a, cache=(batch_step.position_offsets(a["offsets"]), lengths, table))
        T = a["x"].shape[0]
        x = a["x"].double().cpu().numpy()
        ref, tol = x @ Wqkv.T, base_tol(dtype, np.abs(x) @ np.abs(Wqkv).T, SIZE["hidden"])
        assert_near(step.rows[:T].flatten(1), ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, "q|k|v")
        got = step.rows[:T].float().cpu().numpy()
        at = 0
        for r, n in enumerate(new):
            for i, x in enumerate((got[at:at + n, heads:heads + kv], got[at:at + n, heads + kv:])):
                rows[r][i][here[r]:here[r] + n] = x
            at += n
        held = [tuple(values(*stored(x[:here[r] + new[r]], fmt)) for x in rows[r]) for r in range(len(new))]
        check_attention(step.seen[:T], step.rows[:T, :heads], held, here + new, new, heads, kv, dim, dtype, 1, window)
        s = step.seen[:T].flatten(1).double().cpu().numpy()
        ref, tol = s @ Wout.T, base_tol(dtype, np.abs(s) @ np.abs(Wout).T, heads * dim)
        assert_near(step.x[:T], ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, "output projection")
        # the rest is what a step without the layer does with those rows
        plain = batch_step.BatchStep(step.gate_up, step.down, step.head, (step.A, step.B, step.scales), ffn=256, most_tokens=40,
                                     dtype=dtype, **{k: v for k, v in SIZE.items() if k != "n_adapters"})
        want = plain(**dict(a, x=step.x[:T].clone()))
        assert torch.equal(n_accepted, want[0]) and torch.equal(tokens, want[1])
        here = here + n_accepted.cpu().numpy() + 1


def test_a_captured_step_with_a_cache(hq):
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(1810)
    drafted, W = [2, 4, 0], 8
    cache, step = make(g, "bf16", "q4_0", 8, 2, 128, 16, W, 16)
    lengths, table = batch_step.random_cache(g, cache, [100, 60, 90], W)
    fill(g, cache, [100, 60, 90], table)
    inputs = [batch_step.random_inputs(g, drafted, **SIZE) for _ in range(3)]
    offsets = batch_step.position_offsets(inputs[0]["offsets"])
    held = {k: v.clone() for k, v in inputs[0].items()}
    pool = cache.pool.clone()
    step(**held, cache=(offsets, lengths, table))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(**held, cache=(offsets, lengths, table))
    for n, i in enumerate(inputs):
        lengths.copy_(torch.tensor([50 + n, 30 + n, 5 + n], dtype=torch.int32))
        for k, v in held.items():
            v.copy_(i[k])
        cache.pool.copy_(pool)
        want = tuple(v.clone() for v in step(**held, cache=(offsets, lengths, table))), step.logits.clone()
        cache.pool.copy_(pool)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0][0]) and torch.equal(out[1], want[0][1]) and torch.equal(step.logits[:9], want[1][:9])


def test_a_step_refuses_another_cache(hq):
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(1820)
    cache, step = make(g, "bf16", "q8_0", 4, 1, 64, 16, 2, 8)
    lengths, table = batch_step.random_cache(g, cache, [20, 9], 2)
    a = batch_step.random_inputs(g, [1, 2], **SIZE)
    offsets = batch_step.position_offsets(a["offsets"])
    for bad in (None, (offsets[:2], lengths[:1], table[:1]), (offsets, lengths, table.repeat(1, 2)), (offsets.long(), lengths, table)):
        with pytest.raises(ValueError):
            step(**a, cache=bad)
    plain = batch_step.random_step(g, ffn=256, rank=8, most_tokens=8, **SIZE)
    with pytest.raises(ValueError):
        plain(**a, cache=(offsets, lengths, table))
    step(**a, cache=(offsets, lengths, table))
