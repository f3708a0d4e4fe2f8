"""Values at the ends of their range through the batched step, against plain
64-bit statements: infinities and NaN stay where the definition has them."""
from __future__ import annotations

import numpy as np
import pytest

import test_gpu_batch as tb
from quantized_weight_matvec_hq_gb300 import synthetic
from test_gpu_batch import DT, U_OUT, base_tol, dense, dev, exponents, hq, no_device_fault, run_lora, weights  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def assert_same_kind(y, ref, what):
    """Infinities with their signs and NaN exactly where the reference has them."""
    y = y.double().cpu().numpy()
    for name, kind in (("NaN", np.isnan), ("+inf", lambda v: v == np.inf), ("-inf", lambda v: v == -np.inf)):
        wrong = kind(y) != kind(ref)
        assert not wrong.any(), (what, name, np.argwhere(wrong)[:5].tolist(), y[wrong][:5], ref[wrong][:5])


def assert_near_or_same_kind(y, ref, tol, what):
    assert_same_kind(y, ref, what)
    ok = np.isfinite(ref)
    got = y.double().cpu().numpy()
    bad = ok & ~(np.abs(np.where(ok, got, 0) - np.where(ok, ref, 0)) <= np.where(ok, tol, 0))
    assert not bad.any(), (what, np.argwhere(bad)[:5].tolist(), got[bad][:5], ref[bad][:5], tol[bad][:5])


def adapted(hq, fmt, rows, cols, T, n, rank, dtype, seed, spoil=None):
    """A call, the 64-bit result and its tolerance; `spoil` changes x, A, B and the scales before."""
    g = synthetic.rng(seed)
    blocks = weights(g, fmt, rows, cols)
    W = dev(blocks)
    e = exponents(hq, fmt, W, 1, rows, cols)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    A = (torch.from_numpy(g.standard_normal((n, rank, cols)).astype(np.float32)) * 0.05).bfloat16().cuda()
    B = (torch.from_numpy(g.standard_normal((n, rows, rank)).astype(np.float32)) * 0.05).bfloat16().cuda()
    s = dev(g.uniform(0.5, 2, n).astype(np.float32) * np.where(np.arange(n) % 2, -1, 1).astype(np.float32))
    ids = g.integers(-1, n, T)
    ids[:min(T, n + 1)] = np.arange(-1, n)[:min(T, n + 1)]      # every adapter and none, in one tile
    if spoil:
        spoil(x, A, B, s)
    y = run_lora(hq, fmt, W, e, x, dev(ids.astype(np.int32)), A, B, s, n, rank, rows, cols, dtype)
    xd, Wd = x.double().cpu().numpy(), dense(fmt, blocks, rows, cols)
    Ad, Bd, sd = A.double().cpu().numpy(), B.double().cpu().numpy(), s.double().cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        ref, tol = xd @ Wd.T, base_tol(dtype, np.abs(xd) @ np.abs(Wd).T, cols)
        for a in range(n):
            t = np.nonzero(ids == a)[0]
            u, um = xd[t] @ Ad[a].T, np.abs(xd[t]) @ np.abs(Ad[a]).T
            ref[t] += sd[a] * (u @ Bd[a].T)
            # fp32 sums of the columns and of the ranks; u rounded to 16 bits (f32: 24)
            tol[t] += abs(sd[a]) * (um @ np.abs(Bd[a]).T) * ((cols / 8 + 64 + rank) * 2.0 ** -23 + (0 if dtype == "f32" else 2.0 ** -16))
        tol = tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25
    return y, ref, tol, ids


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,rows,cols,T,n,rank", [("q8_0", 300, 1024, 70, 3, 16), ("q4_0", 130, 2048, 5, 3, 5),
                                                    ("q8_0", 77, 512, 9, 4, 64), ("q8_0", 700, 512, 400, 5, 64),
                                                    ("q4_0", 256, 768, 33, 6, 16), ("q8_0", 20000, 256, 40, 3, 5)])
def test_non_finite_adapter_stays_with_its_tokens(hq, fmt, rows, cols, T, n, rank, dtype):
    """Infinities and NaN in one adapter's B reach that adapter's tokens, in
    those rows, and no token of another adapter or of none."""
    def spoil(x, A, B, s):
        B[1, 17, rank - 1] = float("inf")
        B[1, 40, 0] = float("-inf")
        B[1, rows - 1, rank // 2] = float("nan")
        B[1, 5, 1], B[1, 5, 2] = float("inf"), float("-inf")
        B[1, 6, :] = float("inf")
        B[2, 17, 0] = float("inf")
    y, ref, tol, ids = adapted(hq, fmt, rows, cols, T, n, rank, dtype, 300 + rows + rank, spoil)
    assert np.isfinite(ref[ids != 1][:, 18:]).all() and np.isfinite(ref[(ids != 1) & (ids != 2)]).all()
    assert np.isnan(ref[ids == 1][:, -1]).all() and np.isinf(ref[ids == 1][:, 17]).all()
    assert_near_or_same_kind(y, ref, tol, "mixed adapters")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_adapter_leaves_other_tokens_alone(hq, dtype):
    """An infinity in an adapter's A: its tokens' outputs are no numbers or
    infinite, the others as ever."""
    def spoil(x, A, B, s):
        A[1, 3, 100] = float("inf")
    y, ref, tol, ids = adapted(hq, "q8_0", 200, 512, 40, 4, 9, dtype, 330, spoil)
    assert not np.isfinite(ref[ids == 1]).any() and not torch.isfinite(y[dev(ids == 1)]).any()
    assert_near_or_same_kind(y[dev(ids != 1)], ref[ids != 1], tol[ids != 1], "the rest")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_tokens_through_an_adapter(hq, dtype):
    """At rank 1 an infinite element gives infinities of the signs of W and of
    B A, and NaN where the two differ."""
    def spoil(x, A, B, s):
        x[:8, 77] = float("inf")
        x[8:16, 400] = float("-inf")
    y, ref, tol, ids = adapted(hq, "q8_0", 200, 512, 40, 4, 1, dtype, 334, spoil)
    assert np.isinf(ref[:16]).any() and np.isnan(ref[:16]).any()
    assert_near_or_same_kind(y, ref, tol, "infinite tokens")


def test_largest_fp32_tokens_through_an_adapter(hq):
    """Finite fp32 elements above the largest 16-bit brain float: finite
    outputs, near but for what lies 2^-38 below a token's largest element."""
    def spoil(x, A, B, s):
        x[3, 50], x[4, 51] = 3.4e38, -3.4e38
        A[:, :, 50:52] = 1e-20
    y, ref, tol, ids = adapted(hq, "q8_0", 200, 512, 12, 2, 8, "f32", 331, spoil)
    assert ids[3] >= 0 or ids[4] >= 0
    assert np.isfinite(ref).all()
    tol[3:5] += 512 * 2.0 ** -38 * 3.4e38 * 0.25            # weights of deviation 0.02 are below 0.25
    assert_near_or_same_kind(y, ref, tol, "near the largest")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,T", [(140, 37), (130, 200)])
def test_infinite_tokens_have_the_sign_of_their_weights(hq, rows, T, dtype):
    """One infinite element of a token: each output is the infinity of its
    weight's sign, and NaN where that weight is zero."""
    g = synthetic.rng(332 + rows)
    cols = 512
    blocks = weights(g, "q8_0", rows, cols)
    Wd = dense("q8_0", blocks, rows, cols)
    W = dev(blocks)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    x[5, 7], x[20, 300], x[21, 9] = float("nan"), float("inf"), float("-inf")
    y = run_lora(hq, "q8_0", W, exponents(hq, "q8_0", W, 1, rows, cols), x, None, None, None, None, 0, 0, rows, cols, dtype)
    xd = x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = np.where(np.isfinite(xd), xd, 0) @ Wd.T
        for t, j in ((5, 7), (20, 300), (21, 9)):
            ref[t] = ref[t] + xd[t, j] * Wd[:, j]
    assert np.isinf(ref[20]).any()
    assert_same_kind(y, ref, dtype)


@pytest.mark.parametrize("vocab", [50, 9001, 300_000])
def test_softmax_at_the_ends_of_the_temperature(hq, vocab):
    """Infinite and huge temperatures, differences past the largest float,
    masked columns, and a temperature that is no number (greedy)."""
    g = synthetic.rng(333)
    l = g.standard_normal((6, vocab)).astype(np.float32) * 5
    l[:, 3::7] = -np.inf
    l[1, :] = np.where(np.isfinite(l[1]), np.sign(l[1]) * 3e38, -np.inf)
    l[2, :] = np.where(np.isfinite(l[2]), l[2] * 1e37, -np.inf)
    l[5, vocab // 2:] = -np.inf
    t = np.array([np.inf, 1e38, 2e37, 1e-30, np.nan, np.inf], np.float32)
    p = torch.full((6, vocab), float("nan"), device="cuda")
    hq.hq_softmax_rows(dev(l), dev(t), p, 6, vocab, hq.HQ_DT_F32)
    ld, td = l.astype(np.float64), t.astype(np.float64)
    for r in range(6):
        if np.isnan(td[r]):
            ref = (np.arange(vocab) == int(np.argmax(ld[r]))).astype(np.float64)
        else:
            z = (np.where(np.isfinite(ld[r]), ld[r], 0) - ld[r].max()) / td[r]
            ex = np.where(np.isfinite(ld[r]), np.exp(np.maximum(z, -1000)), 0)
            ref = ex / ex.sum()
        # the argument rounded three times (2^-22 of it), power and quotient a few ulps, a sum of rounded terms
        tol = ref * (120 * 2.0 ** -22 + 2.0 ** -19) + 1e-44
        got = p[r].double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), (r, got[:8], ref[:8])


def test_swiglu_of_fp32_tokens_uses_the_accurate_power(hq):
    """Gates that the product gives exactly (one weight and one power of two
    each): z / (1 + e^-z) within 2^-21 for z down to -88, where e^-z is still
    a float (2 ulps of the power, an ulp each for sum, quotient and product)."""
    n, cols = 216, 256
    z = np.arange(n) - 88
    q = np.zeros((2 * n, 8, 34), np.uint8)
    q[:, :, :2] = np.frombuffer(np.float16(1).tobytes(), np.uint8)
    q[0::2, 0, 2] = z.astype(np.int8).view(np.uint8)
    q[1::2, 0, 2] = 1
    q[0::2, 1, 2] = np.where(z > 127, 1, 0)
    q[0::2, 0, 2] = np.where(z > 127, 127, z).astype(np.int8).view(np.uint8)
    W = dev(q.reshape(-1))
    x = torch.zeros((3, cols), device="cuda")
    x[:, 0] = torch.tensor([1.0, 0.25, 2.0 ** -10], device="cuda")
    ids = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    e = exponents(hq, "q8_0", W, 1, 2 * n, cols)
    y = tb.run_moe(hq, W, e, ids, x, 0, None, hq.HQ_MOE_EPI_SWIGLU, 1, 2 * n, cols, "f32")[:, 0].double().cpu().numpy()
    for t, s in enumerate((1.0, 0.25, 2.0 ** -10)):
        zs = np.minimum(z, 127) * s
        ref = zs / (1 + np.exp(-zs)) * s
        assert (np.abs(y[t] - ref) <= 2.0 ** -21 * np.abs(ref)).all(), (s, np.max(np.abs(y[t] - ref) / np.maximum(np.abs(ref), 1e-300)))


def test_output_rows_of_4_gigabytes(hq):
    """2^30 rows of fp32 outputs: the second token's row begins at byte 2^32.
    4-bit weights of one block of columns, 155 GB of them."""
    torch.cuda.empty_cache()
    rows, cols, T = 1 << 30, 256, 2
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("200 GiB of free device memory needed")
    W = torch.zeros((rows, 8, 18), dtype=torch.uint8, device="cuda")        # d = 0: zeros
    at = [0, 1, 77, 1 << 20, (1 << 29) + 5, rows - 1]
    half = torch.tensor(list(np.float16(0.5).tobytes()), dtype=torch.uint8, device="cuda")
    for i, r in enumerate(at):
        W[r, 0, :2] = half
        W[r, 0, 2:] = 0x88                                                  # quants of 0 ...
        W[r, 0, 2] = 0x89 + i                                               # ... but the first: 1 + i
    x = torch.zeros((T, cols), device="cuda")
    x[0, 0], x[1, 0] = 2.0, -3.0
    e = torch.tensor([-11], dtype=torch.int32, device="cuda")               # 8 * 0.5 < 2^(e + 14)
    y = run_lora(hq, "q4_0", W, e, x, None, None, None, None, 0, 0, rows, cols, "f32")
    for i, r in enumerate(at):
        assert y[:, r].tolist() == [1.0 + i, -1.5 * (1 + i)], r
    assert [int(torch.count_nonzero(y[t])) for t in range(T)] == [len(at)] * T
    del W, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("adapters", [0, 2])
def test_weights_written_just_before_the_product(hq, dtype, adapters):
    """Quantizing, the exponents and the product back to back on one stream, and
    the weights rewritten between the replays of a graph."""
    g = synthetic.rng(335)
    rows, cols, T = 1280, 1024, 24
    src = [dev(synthetic.weights(g, rows, cols, s)) for s in (0.02, 0.5, 3.0)]
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    A, B = torch.zeros((2, 4, cols), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, rows, 4), dtype=torch.bfloat16, device="cuda")
    s, ids = torch.ones(2, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    W = torch.empty(rows * cols // 32 * 34, dtype=torch.uint8, device="cuda")
    e = torch.empty(1, dtype=torch.int32, device="cuda")
    w = torch.empty_like(src[0])
    y = torch.empty((T, rows), dtype=DT[dtype], device="cuda")
    ws = tb.dirty(hq.hq_matmul_adapters_workspace(4 if adapters else 0, rows, cols, T, hq.DTYPE_CODES[dtype]))

    def step():
        hq.hq_quantize_q8_0(w, W, rows, cols)
        hq.hq_weight_exponents(8, W, e, 1, rows, cols)
        hq.hq_matmul_q8_0_adapters(W, e, x, ids, A, B, s, adapters, 4, y, rows, cols, T, hq.DTYPE_CODES[dtype], ws, ws.numel())

    want = []
    for m in src:
        w.copy_(m)
        hq.hq_quantize_q8_0(w, W, rows, cols)
        torch.cuda.synchronize()
        Wd = dense("q8_0", W.cpu().numpy(), rows, cols)
        xd = x.double().cpu().numpy()
        want.append((xd @ Wd.T, base_tol(dtype, np.abs(xd) @ np.abs(Wd).T, cols)))

    def check(i):
        ref, tol = want[i]
        tb.assert_near(y, ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, f"weights {i}")
    for i in (0, 1, 2, 0):
        w.copy_(src[i])
        step()
        check(i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in (1, 2, 0, 1):
        w.copy_(src[i])
        graph.replay()
        check(i)
