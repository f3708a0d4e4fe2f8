"""GPU tests of the batched step as a whole, and of the many-token calls where
their inner paths change: many slots, many adapters a window, shared token
tiles, weights of very different sizes in one matrix, extreme temperatures.

Tolerances are those of the single calls (see test_gpu_batch.py), each stage
against the 64-bit form of its own inputs.
"""
from __future__ import annotations

import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import synthetic
from test_gpu_batch import (U_OUT, DT, assert_near, base_tol, check_moe, dense, dev, exponents, hq, lora_case,  # noqa: F401
                            moe_reference, no_device_fault, run_moe, softmax_reference, verify_reference, weights)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_step(hq, dtype):
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(900)
    size = dict(n_experts=8, n_active=3, hidden=512, vocab=2050, n_adapters=4, dtype=dtype)
    ffn, rank, drafted = 256, 12, [3, 0, 5, 1, 1, 7, 0, 2]
    step = batch_step.random_step(g, ffn=ffn, rank=rank, most_tokens=40, **size)
    a = batch_step.random_inputs(g, drafted, **size)
    n_accepted, tokens = step(**a)
    T, E, k, hid, V = a["x"].shape[0], 8, 3, 512, 2050

    def bank(blocks, rows, cols, mats=1):
        return dense("q8_0", blocks.cpu().numpy(), mats * rows, cols).reshape(mats, rows, cols)
    ids, rw = a["expert_ids"].cpu().numpy(), a["router_w"].cpu().numpy().astype(np.float64)
    ref, mag = moe_reference(bank(step.gate_up, 2 * ffn, hid, E), ids, a["x"].double().cpu().numpy(), None, 1, 0)
    check_moe(step.h[:T], ref, mag, None, 1, dtype, hid, "gate|up")
    ref, mag = moe_reference(bank(step.down, hid, ffn, E), ids, step.h[:T].double().cpu().numpy(), None, 2, 1)
    check_moe(step.y[:T], ref, mag, rw, 2, dtype, ffn, "down")

    y, W = step.y[:T].double().cpu().numpy(), bank(step.head, V, hid)[0]
    ref, tol = y @ W.T, base_tol(dtype, np.abs(y) @ np.abs(W).T, hid)
    A, B = step.A.double().cpu().numpy(), step.B.double().cpu().numpy()
    for t, ad in enumerate(a["adapter_ids"].cpu().numpy()):
        if ad >= 0:
            s = float(step.scales[ad])
            ref[t] += s * (B[ad] @ (A[ad] @ y[t]))
            tol[t] += abs(s) * (np.abs(B[ad]) @ (np.abs(A[ad]) @ np.abs(y[t]))) * \
                ((hid / 8 + 64 + rank) * 2.0 ** -23 + (0 if dtype == "f32" else 2.0 ** -16))
    assert_near(step.logits[:T], ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, "logits")

    l, t = step.logits[:T].double().cpu().numpy(), a["temperature"].cpu().numpy().astype(np.float64)
    p = softmax_reference(l, t)
    z = (l.max(1, keepdims=True) - l) / np.where(t > 0, t, 1)[:, None]
    assert_near(step.p[:T], p, p * (np.minimum(z, 120) * 2.0 ** -22 + 2.0 ** -19) + 1e-44, "probabilities")
    want = verify_reference(step.p[:T].cpu().numpy(), None, a["drafts"].cpu().numpy(), a["offsets"].cpu().numpy(),
                            a["u_accept"].cpu().numpy(), a["u_sample"].cpu().numpy())
    assert np.array_equal(n_accepted.cpu().numpy(), want[0]) and np.array_equal(tokens.cpu().numpy(), want[1])


def test_step_in_a_graph(hq):
    """Captured, and replayed with new inputs: the tokens of a plain call."""
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(901)
    size = dict(n_experts=16, n_active=2, hidden=256, vocab=1000, n_adapters=2)
    step = batch_step.random_step(g, ffn=256, rank=8, most_tokens=16, **size)
    drafted = [2, 4, 0, 3]
    inputs = [batch_step.random_inputs(g, drafted, **size) for _ in range(3)]
    want = [tuple(v.clone() for v in step(**i)) for i in inputs]
    torch.cuda.synchronize()
    held = {k: v.clone() for k, v in inputs[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(**held)
    for i, w in zip(inputs, want):
        for k, v in held.items():
            v.copy_(i[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])


def test_step_refuses_wrong_sizes(hq):
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = synthetic.rng(902)
    size = dict(n_experts=4, n_active=1, hidden=256, vocab=64, n_adapters=1)
    step = batch_step.random_step(g, ffn=256, rank=1, most_tokens=4, **size)
    with pytest.raises(ValueError):
        step(**batch_step.random_inputs(g, [3, 1], **size))           # six positions of four
    a = batch_step.random_inputs(g, [1, 1], **size)
    with pytest.raises(ValueError):
        step(**dict(a, drafts=a["drafts"][:1]))
    step(**a)


@pytest.mark.parametrize("dtype,T,k,E,per_slot", [("bf16", 1100, 8, 16, 0), ("f16", 2900, 3, 5, 1), ("f32", 1030, 8, 64, 0)])
def test_moe_of_many_slots(hq, dtype, T, k, E, per_slot):
    """More slots than one block places (8192), and one expert without any."""
    g = synthetic.rng(910 + T)
    rows, cols = 40, 256
    blocks = weights(g, "q8_0", E * rows, cols)
    Wd, W = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols), dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    ids = g.integers(0, E - 1, (T, k)).astype(np.int32)
    x = torch.from_numpy(g.standard_normal((T, k, cols) if per_slot else (T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    ref, mag = moe_reference(Wd, ids, x.double().cpu().numpy(), None, 0, per_slot)
    y = run_moe(hq, W, e, dev(ids), x, per_slot, None, 0, E, rows, cols, dtype)
    check_moe(y, ref, mag, None, 0, dtype, cols, "many slots")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,rows,cols,T,n,rank", [("q8_0", 96, 256, 400, 130, 5), ("q4_0", 200, 512, 129, 129, 64),
                                                    ("q8_0", 640, 1024, 230, 3, 20), ("q8_0", 129, 2048, 8, 8, 40)])
def test_many_adapters_and_shared_tiles(hq, fmt, rows, cols, T, n, rank, dtype):
    """An adapter a token; windows of tokens that end inside the batch; an odd number of row tiles."""
    g = synthetic.rng(920 + rows)
    ids = g.permutation(T) % n
    ids[::11] = -1
    y, ref, tol = lora_case(hq, fmt, rows, cols, T, n, rank, dtype, 921 + rows, ids)
    assert_near(y, ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, "adapters")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_matrix_of_large_and_small_weights(hq, dtype):
    """Rows from 1 to 2^-30 of the largest.  16 bits: what is left of a weight is within 2^-11 of it or 2^-22 of the
    matrix's largest (a decoded weight and its block's offset are rounded to 2^-24, the largest is above 0.24);
    f32: 2^-36 of it."""
    g = synthetic.rng(930)
    rows, cols, T = 93, 512, 21
    w = synthetic.weights(g, rows, cols, 1.0) * 2.0 ** -np.arange(rows)[:, None].clip(0, 30).astype(np.float32)
    import oracle
    blocks = oracle.quantize("q8_0", w).reshape(-1)
    Wd, W = dense("q8_0", blocks, rows, cols)[None], dev(blocks)
    e = exponents(hq, "q8_0", W, 1, rows, cols)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    xd = x.double().cpu().numpy()
    ids = np.zeros((T, 1), np.int32)
    ref, mag = moe_reference(Wd, ids, xd, None, 0, 0)
    y = run_moe(hq, W, e, dev(ids), x, 0, None, 0, 1, rows, cols, dtype)
    floor = np.abs(Wd).max() * np.abs(xd).sum(1)[:, None, None] * (2.0 ** -36 if dtype == "f32" else 2.0 ** -22)
    tol = base_tol(dtype, mag, cols) + floor
    assert_near(y, ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, "wide range")


def test_softmax_of_extreme_temperatures(hq):
    """From sharper than any difference of logits to flat, with -inf, the type's lowest value and a NaN row."""
    g = synthetic.rng(940)
    t = np.array([1e-38, 1e-20, 1e-18, 1e-6, 1.0, 30.0, 1e17, 1e18, 1e30, 3e38, 0.7], np.float32)
    V = 20_011
    x = (g.standard_normal((len(t), V)) * 10).astype(np.float32)
    x[:, 3::7] = -np.inf
    x[:, 5::7] = np.finfo(np.float32).min
    x[10, 8] = np.nan
    p = torch.full((len(t), V), float("nan"), device="cuda")
    hq.hq_softmax_rows(dev(x), dev(t), p, len(t), V, hq.HQ_DT_F32)
    l, td = x.astype(np.float64), t.astype(np.float64)
    # the difference of two logits is rounded once to fp32, as the argument of the power is
    with np.errstate(invalid="ignore", over="ignore"):
        ref = softmax_reference(l, td)
        z = np.where(np.isfinite(l), np.nanmax(np.where(np.isfinite(l), l, -np.inf), axis=1, keepdims=True) - l, 0) / td[:, None]
    assert np.isnan(p[10].cpu().numpy()).all()
    tol = ref * (np.minimum(z, 120) * 2.0 ** -22 + 2.0 ** -19) + 1e-44
    assert_near(p[:10], ref[:10], tol[:10], "extreme temperatures")
