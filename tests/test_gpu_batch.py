"""GPU parity of the batched step (grouped and adapted products of many tokens,
softmax rows, draft verification) against plain 64-bit statements.

Tolerance of the 16-bit products, per output, with T = sum |w x|: each weight
is rounded to 11 bits (2^-11 of each term, worst case), the fp32 sums of the
tensor core round once per 16 columns (2^-22 each, whatever its rounding
mode), and y is rounded once (u = 2^-11 f16, 2^-8 bf16, taken a bit wide).
The f32 products drop a term of 2^-21 |w x| at most, both splits leave 2^-22,
and the sums leave the tensor core every 256 columns: 48 additions of 2^-22.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from quantized_weight_matvec_hq_gb300 import synthetic

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U_OUT = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}
BYTES = {"q8_0": 34, "q4_0": 18}


@pytest.fixture(scope="module")
def hq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_matvec_hq_gb300 import build
    build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    return hq


@pytest.fixture(autouse=True)
def no_device_fault(hq):
    yield
    assert hq.hq_device_fault() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def base_tol(dtype, T, cols):
    if dtype == "f32":
        return T * (2.0 ** -20 + 48 * 2.0 ** -22 + (cols / 256) * 2.0 ** -23)
    return T * (2.0 ** -11 + (cols / 16 + 8) * 2.0 ** -22)


def assert_near(y, ref, tol, what):
    y = y.double().cpu().numpy()
    assert y.shape == ref.shape
    bad = ~(np.abs(y - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(y - ref) - tol, -1)), ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of tolerance; at {i}: {y[i]!r}, ref {ref[i]!r}, tol {tol[i]!r}")


def weights(g, fmt, rows, cols, std=0.02):
    return oracle.quantize(fmt, synthetic.weights(g, rows, cols, std)).reshape(-1)


def dense(fmt, blocks, rows, cols):
    return oracle.dequant(fmt, blocks, rows, cols).astype(np.float64).reshape(rows, cols)


def exponents(hq, fmt, W, n_mats, rows, cols):
    e = torch.full((n_mats,), 99, dtype=torch.int32, device="cuda")
    hq.hq_weight_exponents(hq.FMT_CODES[fmt], W, e, n_mats, rows, cols)
    return e


def dirty(n):
    return torch.full((max(int(n), 1),), 0xFF, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ set-up

def test_weight_exponents(hq):
    g = synthetic.rng(40)
    for fmt, top in (("q8_0", 128.0), ("q4_0", 8.0)):
        mats = [weights(g, fmt, 33, 320, s) for s in (0.02, 1e-6, 300.0, 1.0)]
        z = mats[3].copy().reshape(33, -1, BYTES[fmt])
        z[..., :2] = 0
        z[5, 3, :2] = np.frombuffer(np.float16(np.inf).tobytes(), np.uint8)
        z[6, 1, :2] = np.frombuffer(np.float16(-0.5).tobytes(), np.uint8)
        mats[3] = z.reshape(-1)
        mats.append(np.zeros_like(z).reshape(-1))
        e = exponents(hq, fmt, dev(np.concatenate(mats)), len(mats), 33, 320).cpu().numpy()
        for i, m in enumerate(mats):
            d = np.abs(np.ascontiguousarray(m.reshape(-1, BYTES[fmt])[:, :2]).view(np.float16).astype(np.float64))
            d = d[np.isfinite(d)].max()
            assert e[i] == (np.frexp(d * top)[1] - 14 if d else -14), (fmt, i)
            with np.errstate(invalid="ignore"):
                w = np.abs(dense(fmt, m, 33, 320))
            assert w[np.isfinite(w)].max() < 2.0 ** (e[i] + 14)


# ------------------------------------------------------------------ grouped products

def moe_reference(Wd, ids, x, w_router, epi, per_slot):
    """f64 result and the magnitudes that bound its error."""
    T, k = ids.shape
    E, rows, cols = Wd.shape
    y, mag = np.zeros((T, k, rows)), np.zeros((T, k, rows))
    for e in range(E):
        t, s = np.nonzero(ids == e)
        if len(t):
            xe = x[t, s] if per_slot else x[t]
            y[t, s] = xe @ Wd[e].T
            mag[t, s] = np.abs(xe) @ np.abs(Wd[e]).T
    return y, mag


def run_moe(hq, W, e, ids, x, per_slot, rw, epi, E, rows, cols, dtype, stream=None, ws=None):
    T, k = ids.shape
    shape = {0: (T, k, rows), 1: (T, k, rows // 2), 2: (T, rows)}[epi]
    y = torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda")
    n = hq.hq_moe_matmul_workspace(E, k, rows, cols, T, per_slot, hq.DTYPE_CODES[dtype], epi)
    ws = dirty(n) if ws is None else ws
    assert ws.numel() >= n
    hq.hq_moe_matmul_q8_0(W, e, ids, x, per_slot, rw, y, E, k, rows, cols, T, hq.DTYPE_CODES[dtype], epi, ws, ws.numel(),
                          stream=stream)
    return y


def check_moe(y, ref, mag, rw, epi, dtype, cols, what):
    tol = base_tol(dtype, mag, cols)
    if epi == 1:
        gt, ut, ge, ue = ref[..., 0::2], ref[..., 1::2], tol[..., 0::2], tol[..., 1::2]
        h = gt / (1 + np.exp(-gt)) * ut
        sg = np.abs(gt / (1 + np.exp(-gt)))
        t = 1.1 * ge * (np.abs(ut) + ue) + sg * ue + 1e-6 * (sg + 1.1 * ge) * (np.abs(ut) + ue)
        assert_near(y, h, t + U_OUT[dtype] * (np.abs(h) + t) + 2.0 ** -25, what)
    elif epi == 2:
        c = np.einsum("tkr,tk->tr", ref, rw)
        t = np.einsum("tkr,tk->tr", tol + 2.0 ** -21 * np.abs(ref), np.abs(rw))
        assert_near(y, c, t + U_OUT[dtype] * (np.abs(c) + t) + 2.0 ** -25, what)
    else:
        assert_near(y, ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, what)


# (experts, active, rows, cols, tokens, x per slot)
MOE_SHAPES = [(1, 1, 1, 256, 1, 0), (4, 2, 77, 256, 3, 1), (8, 3, 130, 512, 40, 0), (16, 8, 256, 768, 33, 1),
              (3, 1, 384, 1280, 517, 0), (61, 5, 62, 2048, 97, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("E,k,rows,cols,T,per_slot", MOE_SHAPES)
def test_moe_parity(hq, E, k, rows, cols, T, per_slot, dtype):
    g = synthetic.rng(1000 + E + rows)
    blocks = weights(g, "q8_0", E * rows, cols)
    Wd = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    ids = synthetic.expert_ids(g, T, k, E)
    x = torch.from_numpy(g.standard_normal((T, k, cols) if per_slot else (T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    rw = synthetic.router_weights(g, T, k)
    ref, mag = moe_reference(Wd, ids, x.double().cpu().numpy(), rw, 0, per_slot)
    for epi in (0, 1, 2):
        if epi == 1 and rows % 2:
            continue
        y = run_moe(hq, W, e, dev(ids), x, per_slot, dev(rw), epi, E, rows, cols, dtype)
        check_moe(y, ref, mag, rw, epi, dtype, cols, f"epilogue {epi}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_ragged_extremes(hq, dtype):
    """Every token at one expert; the first and last expert only; groups around
    the sizes at which a tile ends."""
    g = synthetic.rng(51)
    E, rows, cols = 9, 200, 512
    blocks = weights(g, "q8_0", E * rows, cols)
    Wd = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    sizes = [[0, 0, 300, 0, 0, 0, 0, 0, 0], [1, 0, 0, 0, 0, 0, 0, 0, 1], [16, 17, 15, 32, 33, 64, 65, 63, 31],
             [128, 129, 127, 0, 256, 257, 255, 1, 2]]
    for s in sizes:
        ids = g.permutation(np.repeat(np.arange(E), s)).astype(np.int32)[:, None]
        x = torch.from_numpy(g.standard_normal((len(ids), cols)).astype(np.float32)).cuda().to(DT[dtype])
        ref, mag = moe_reference(Wd, ids, x.double().cpu().numpy(), None, 0, 0)
        y = run_moe(hq, W, e, dev(ids), x, 0, None, 0, E, rows, cols, dtype)
        check_moe(y, ref, mag, None, 0, dtype, cols, f"groups {s}")


def test_moe_duplicate_experts_of_one_token(hq):
    g = synthetic.rng(52)
    E, k, rows, cols, T = 4, 4, 66, 256, 21
    blocks = weights(g, "q8_0", E * rows, cols)
    Wd = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    ids = g.integers(0, 2, size=(T, k)).astype(np.int32)
    x = torch.from_numpy(g.standard_normal((T, k, cols)).astype(np.float32)).cuda().bfloat16()
    rw = synthetic.router_weights(g, T, k)
    ref, mag = moe_reference(Wd, ids, x.double().cpu().numpy(), rw, 2, 1)
    y = run_moe(hq, W, e, dev(ids), x, 1, dev(rw), 2, E, rows, cols, "bf16")
    check_moe(y, ref, mag, rw, 2, "bf16", cols, "duplicates")


@pytest.mark.parametrize("epi", [0, 1, 2])
def test_moe_invalid_ids(hq, epi):
    """NaN for the slots of an id out of range (for the whole token in the
    combine), every other output as usual, and the fault bit."""
    g = synthetic.rng(53)
    E, k, rows, cols, T = 5, 2, 130, 256, 19
    blocks = weights(g, "q8_0", E * rows, cols)
    Wd = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    ids = synthetic.expert_ids(g, T, k, E)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().bfloat16()
    rw = synthetic.router_weights(g, T, k)
    ref, mag = moe_reference(Wd, ids, x.double().cpu().numpy(), rw, 0, 0)
    bad = ids.copy()
    bad[3, 1], bad[18, 0], bad[7, 0] = -1, E, 2 ** 31 - 1
    y = run_moe(hq, W, e, dev(bad), x, 0, dev(rw), epi, E, rows, cols, "bf16")
    assert hq.hq_device_fault() & 0xFF == hq.HQ_FAULT_EXPERT_ID
    wrong = np.zeros((T, k), bool)
    wrong[3, 1] = wrong[18, 0] = wrong[7, 0] = True
    if epi == 2:
        wrong = wrong.any(1)
        assert torch.isnan(y[dev(wrong)]).all()
        check_moe(y[dev(~wrong)], ref[~wrong], mag[~wrong], rw[~wrong], 2, "bf16", cols, "the rest")
    else:
        assert torch.isnan(y[dev(wrong)]).all()
        check_moe(y[dev(~wrong)], ref[~wrong], mag[~wrong], None, epi, "bf16", cols, "the rest")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_moe_equal_runs_streams_and_graph(hq, dtype):
    """The same bits on every run, on another stream, and replayed from a graph
    with new inputs; the workspace's old content never matters."""
    g = synthetic.rng(54)
    E, k, rows, cols, T = 16, 4, 320, 1024, 150
    blocks = weights(g, "q8_0", E * rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    ids = dev(synthetic.expert_ids(g, T, k, E))
    rw = dev(synthetic.router_weights(g, T, k))
    xs = [torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype]) for _ in range(2)]
    first = [run_moe(hq, W, e, ids, x, 0, rw, 2, E, rows, cols, dtype) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = run_moe(hq, W, e, ids, xs[0], 0, rw, 2, E, rows, cols, dtype)
    s.synchronize()
    assert torch.equal(first[0], again)
    x = xs[0].clone()
    y = torch.empty_like(first[0])
    ws = dirty(hq.hq_moe_matmul_workspace(E, k, rows, cols, T, 0, hq.DTYPE_CODES[dtype], 2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        hq.hq_moe_matmul_q8_0(W, e, ids, x, 0, rw, y, E, k, rows, cols, T, hq.DTYPE_CODES[dtype], 2, ws, ws.numel())
    for i in (1, 0, 1):
        x.copy_(xs[i])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first[i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_of_weights_and_tokens(hq, dtype):
    """Experts of weights from 1e-6 to 1e3 and tokens from 1e-30 to 1e30 in one
    call, one element far above the rest of its token, zero tokens."""
    g = synthetic.rng(55)
    E, rows, cols = 4, 96, 512
    mats = [weights(g, "q8_0", rows, cols, s) for s in (2e-6, 0.02, 30.0, 300.0)]
    blocks = np.concatenate(mats)
    Wd = dense("q8_0", blocks, E * rows, cols).reshape(E, rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, E, rows, cols)
    x = g.standard_normal((24, cols)).astype(np.float32)
    x[0:4] *= 1e-30
    x[4:8] *= 1e30
    x[8:12, 100] = 3e4
    x[12] = 0
    ids = (np.arange(24) % 4).astype(np.int32)[:, None]
    xt = torch.from_numpy(x).cuda().to(DT[dtype])
    ref, mag = moe_reference(Wd, ids, xt.double().cpu().numpy(), None, 0, 0)
    y = run_moe(hq, W, e, dev(ids), xt, 0, None, 0, E, rows, cols, dtype).double().cpu().numpy()
    # no absolute floor here: the bound scales with each token; an element 2^-29 below its
    # token's largest may lose 2^-40 of that largest
    wmax = np.abs(Wd).max(axis=(1, 2))[ids[:, 0]][:, None, None]
    floor = cols * 2.0 ** -38 * np.abs(xt.double().cpu().numpy()).max(1)[:, None, None] * wmax
    tol = base_tol(dtype, mag, cols) + floor
    tol = tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -133
    assert (np.abs(y - ref) <= tol).all()
    assert (y[12] == 0).all()


def test_non_finite_tokens_stay_in_their_rows(hq):
    g = synthetic.rng(56)
    rows, cols, T = 140, 512, 37
    for dtype in ("bf16", "f16", "f32"):
        blocks = weights(g, "q8_0", rows, cols)
        W = dev(blocks)
        e = exponents(hq, "q8_0", W, 1, rows, cols)
        x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
        x[5, 7] = float("nan")
        x[20, 300] = float("inf")
        y = torch.empty((T, rows), dtype=DT[dtype], device="cuda")
        ws = dirty(hq.hq_matmul_adapters_workspace(0, rows, cols, T, hq.DTYPE_CODES[dtype]))
        hq.hq_matmul_q8_0_adapters(W, e, x, None, None, None, None, 0, 0, y, rows, cols, T, hq.DTYPE_CODES[dtype], ws,
                                   ws.numel())
        assert torch.isnan(y[5]).all()
        w = dense("q8_0", blocks, rows, cols)[:, 300]
        assert not torch.isfinite(y[20][dev(w != 0)]).any()
        keep = [t for t in range(T) if t not in (5, 20)]
        xs = x[keep].double().cpu().numpy()
        Wd = dense("q8_0", blocks, rows, cols)
        mag = np.abs(xs) @ np.abs(Wd).T
        tol = base_tol(dtype, mag, cols)
        ref = xs @ Wd.T
        assert_near(y[keep], ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, dtype)


# ------------------------------------------------------------------ adapters

def run_lora(hq, fmt, W, e, x, ids, A, B, s, n, rank, rows, cols, dtype):
    T = x.shape[0]
    y = torch.full((T, rows), float("nan"), dtype=DT[dtype], device="cuda")
    ws = dirty(hq.hq_matmul_adapters_workspace(rank, rows, cols, T, hq.DTYPE_CODES[dtype]))
    fn = hq.hq_matmul_q8_0_adapters if fmt == "q8_0" else hq.hq_matmul_q4_0_adapters
    fn(W, e, x, ids, A, B, s, n, rank, y, rows, cols, T, hq.DTYPE_CODES[dtype], ws, ws.numel())
    return y


def lora_case(hq, fmt, rows, cols, T, n, rank, dtype, seed, ids):
    g = synthetic.rng(seed)
    blocks = weights(g, fmt, rows, cols)
    W = dev(blocks)
    e = exponents(hq, fmt, W, 1, rows, cols)
    A = (torch.from_numpy(g.standard_normal((n, rank, cols)).astype(np.float32)) * 0.05).bfloat16().cuda()
    B = (torch.from_numpy(g.standard_normal((n, rows, rank)).astype(np.float32)) * 0.05).bfloat16().cuda()
    s = g.uniform(-2, 2, n).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().to(DT[dtype])
    y = run_lora(hq, fmt, W, e, x, dev(ids.astype(np.int32)), A, B, dev(s), n, rank, rows, cols, dtype)
    xd, Wd = x.double().cpu().numpy(), dense(fmt, blocks, rows, cols)
    ref, tol = xd @ Wd.T, base_tol(dtype, np.abs(xd) @ np.abs(Wd).T, cols)
    Ad, Bd = A.double().cpu().numpy(), B.double().cpu().numpy()
    for a in range(n):
        t = np.nonzero(ids == a)[0]
        if len(t):
            u = xd[t] @ Ad[a].T
            um = np.abs(xd[t]) @ np.abs(Ad[a]).T
            ref[t] += s[a] * (u @ Bd[a].T)
            # fp32 sums of the columns and of the ranks
            tol[t] += abs(s[a]) * (um @ np.abs(Bd[a]).T) * (cols / 8 + 64 + rank) * 2.0 ** -23
    return y, ref, tol


# (format, rows, cols, tokens, adapters, rank)
LORA_SHAPES = [("q8_0", 1, 256, 1, 1, 1), ("q8_0", 77, 512, 5, 3, 8), ("q4_0", 130, 1024, 33, 4, 16),
               ("q8_0", 256, 2048, 64, 64, 16), ("q4_0", 640, 512, 300, 5, 64), ("q8_0", 384, 768, 517, 2, 57),
               ("q4_0", 100, 4096, 2, 2, 33)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,rows,cols,T,n,rank", LORA_SHAPES)
def test_adapters_parity(hq, fmt, rows, cols, T, n, rank, dtype):
    g = synthetic.rng(7000 + rows)
    for kind in ("runs", "mixed"):
        ids = np.sort(g.integers(-1, n, T)) if kind == "runs" else g.integers(-1, n, T)
        y, ref, tol = lora_case(hq, fmt, rows, cols, T, n, rank, dtype, 7100 + rows, ids)
        assert_near(y, ref, tol + U_OUT[dtype] * (np.abs(ref) + tol) + 2.0 ** -25, kind)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_no_adapters_is_the_bare_product(hq, fmt):
    """n_adapters = 0 and ids of -1 give the same bits."""
    g = synthetic.rng(71)
    rows, cols, T = 300, 1024, 70
    blocks = weights(g, fmt, rows, cols)
    W = dev(blocks)
    e = exponents(hq, fmt, W, 1, rows, cols)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().bfloat16()
    bare = run_lora(hq, fmt, W, e, x, None, None, None, None, 0, 0, rows, cols, "bf16")
    A = torch.full((1, 8, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    B = torch.full((1, rows, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    y = run_lora(hq, fmt, W, e, x, ids, A, B, torch.ones(1, device="cuda"), 1, 8, rows, cols, "bf16")
    assert torch.equal(bare, y)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_slow_outputs_do_not_disturb_the_products(hq, fmt):
    """Rank-64 adapters of zeros over several tiles per CTA: the adapter term keeps
    the load unit busy while later tiles are decoded.  Every run has the bits of
    the bare product."""
    g = synthetic.rng(75)
    rows, cols, T, n = 6144, 1024, 2011, 8
    blocks = weights(g, fmt, rows, cols)
    W = dev(blocks)
    e = exponents(hq, fmt, W, 1, rows, cols)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().half()
    A = torch.from_numpy(g.standard_normal((n, 64, cols)).astype(np.float32)).cuda().bfloat16()
    B = torch.zeros((n, rows, 64), dtype=torch.bfloat16, device="cuda")
    ids = dev(np.sort(g.integers(0, n, T)).astype(np.int32))
    bare = run_lora(hq, fmt, W, e, x, None, None, None, None, 0, 0, rows, cols, "f16")
    for _ in range(10):
        y = run_lora(hq, fmt, W, e, x, ids, A, B, torch.ones(n, device="cuda"), n, 64, rows, cols, "f16")
        assert torch.equal(bare, y)


def test_adapter_ids_out_of_range(hq):
    g = synthetic.rng(72)
    ids = g.integers(-1, 3, 50)
    bad = ids.copy()
    bad[4], bad[49] = 3, -2
    y, ref, tol = lora_case(hq, "q8_0", 200, 512, 50, 3, 16, "bf16", 7200, bad)
    assert hq.hq_device_fault() & 0xFF == hq.HQ_FAULT_ADAPTER_ID
    keep = [t for t in range(50) if t not in (4, 49)]
    assert torch.isnan(y[[4, 49]]).all()
    assert_near(y[keep], ref[keep], (tol + 2.0 ** -7 * (np.abs(ref) + tol) + 2.0 ** -25)[keep], "the rest")


def test_row_does_not_depend_on_its_neighbours(hq):
    """A token's row has the same bits wherever it stands among other tokens of the call."""
    g = synthetic.rng(73)
    rows, cols, T = 256, 1024, 130
    blocks = weights(g, "q8_0", rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q8_0", W, 1, rows, cols)
    x = torch.from_numpy(g.standard_normal((T, cols)).astype(np.float32)).cuda().bfloat16()
    perm = torch.from_numpy(g.permutation(T)).cuda()
    a = run_lora(hq, "q8_0", W, e, x, None, None, None, None, 0, 0, rows, cols, "bf16")
    b = run_lora(hq, "q8_0", W, e, x[perm].contiguous(), None, None, None, None, 0, 0, rows, cols, "bf16")
    assert torch.equal(a[perm], b)


def test_products_past_32_bit_offsets(hq):
    """Outputs past 2^31 elements: sampled tokens against the same tokens alone."""
    rows, cols, T = 16384, 256, 140_000
    g = synthetic.rng(74)
    blocks = weights(g, "q4_0", rows, cols)
    W = dev(blocks)
    e = exponents(hq, "q4_0", W, 1, rows, cols)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, cols), generator=gen, device="cuda").bfloat16()
    y = run_lora(hq, "q4_0", W, e, x, None, None, None, None, 0, 0, rows, cols, "bf16")
    Wd = dense("q4_0", blocks, rows, cols)
    for t in (0, 70_001, 131_071, 131_072, T - 1):
        xd = x[t:t + 1].double().cpu().numpy()
        ref, mag = xd @ Wd.T, np.abs(xd) @ np.abs(Wd).T
        tol = base_tol("bf16", mag, cols)
        assert_near(y[t:t + 1], ref, tol + 2.0 ** -7 * (np.abs(ref) + tol) + 2.0 ** -25, f"token {t}")


# ------------------------------------------------------------------ softmax

def softmax_reference(l, t):
    p = np.zeros_like(l)
    for i in range(len(l)):
        if not t[i] > 0:
            v = np.where(np.isnan(l[i]), -np.inf, l[i])
            if v.max() > -np.inf:
                p[i, int(np.argmax(v))] = 1
        elif np.isnan(l[i]).any() or (l[i] == np.inf).any():
            p[i] = np.nan
        elif (l[i] > -np.inf).any():
            ex = np.exp((l[i] - l[i].max()) / t[i])
            p[i] = ex / ex.sum()
    return p


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 31), (5, 1000), (2, 4097), (7, 32003), (3, 151936), (2, 600_001)])
def test_softmax_rows(hq, dtype, rows, vocab):
    g = synthetic.rng(80 + vocab)
    x = torch.from_numpy((g.standard_normal((rows, vocab)) * 4).astype(np.float32)).cuda().to(DT[dtype])
    x[:, ::5] = float("-inf")
    x[:, 0] = 0.25
    if rows > 2:
        x[1] = float("-inf")                              # nothing left
        x[2, vocab // 2:] = torch.finfo(DT[dtype]).min    # the type's lowest value
    t = g.uniform(0.2, 3.0, rows).astype(np.float32)
    if rows > 4:
        t[3], t[4] = 0.0, -1.0
    for temp in (None, t):
        p = torch.full((rows, vocab), float("nan"), device="cuda")
        hq.hq_softmax_rows(x, None if temp is None else dev(temp), p, rows, vocab, hq.DTYPE_CODES[dtype])
        l = x.double().cpu().numpy()
        tt = np.ones(rows) if temp is None else temp.astype(np.float64)
        with np.errstate(over="ignore", invalid="ignore"):
            ref = softmax_reference(l, tt)
            z = np.where(np.isfinite(l), np.abs(l - l[np.isfinite(l)].max()), 0)
        # exponent argument rounded twice (2^-23 of it), exp and quotient a few ulps, a sum of rounded terms
        tol = ref * (np.minimum(z / np.where(tt > 0, tt, 1)[:, None], 120) * 2.0 ** -22 + 2.0 ** -19) + 1e-44
        assert_near(p, ref, tol, f"temperature {temp is not None}")


def test_softmax_in_place_ties_and_non_finite(hq):
    x = torch.zeros((6, 777), device="cuda")
    x[0, 5] = x[0, 700] = 3.0
    x[1, 9] = float("nan")
    x[2, 9] = float("inf")
    x[3] = float("nan")
    x[4, 0] = float("nan")
    x[4, 77] = 1.0
    t = torch.tensor([0.0, 1.0, 1.0, 0.0, 0.0, 1.0], device="cuda")
    hq.hq_softmax_rows(x, t, x, 6, 777, hq.HQ_DT_F32)
    p = x.cpu().numpy()
    assert p[0, 5] == 1 and p[0].sum() == 1
    assert np.isnan(p[1]).all() and np.isnan(p[2]).all()
    assert (p[3] == 0).all()
    assert p[4, 77] == 1 and p[4].sum() == 1
    assert np.allclose(p[5], 1 / 777, rtol=1e-6)


# ------------------------------------------------------------------ verification

def verify_reference(p, q, drafts, off, u, us):
    """The rule on exact integers (numpy float32 for the two rounded operations)."""
    acc, tokens = [], []
    for r in range(len(off) - 1):
        n, a = off[r + 1] - off[r], 0
        V = p.shape[1]
        while a < n:
            i, d = off[r] + a, drafts[off[r] + a]
            if not 0 <= d < V or not np.float32(u[i]) * (q[i, d] if q is not None else np.float32(1)) < p[i + r, d]:
                break
            a += 1
        row = p[off[r] + r + a]
        left = row
        if a < n:
            if q is not None:
                left = row - q[off[r] + a]
            else:
                left = row.copy()
                if 0 <= drafts[off[r] + a] < V:
                    left[drafts[off[r] + a]] -= np.float32(1)
        def ints(s):
            s = np.clip(np.nan_to_num(s.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)
            return [int(v) for v in np.floor(s * 2.0 ** 40)]
        S = ints(left)
        if sum(S) == 0:
            S = ints(row)
        pick = -1
        if sum(S):
            goal = sum(S) * int(np.floor(np.float32(us[r]) * np.float32(2 ** 24))) >> 24
            run = 0
            for j, v in enumerate(S):
                run += v
                if run > goal:
                    pick = j
                    break
        acc.append(a)
        tokens += list(drafts[off[r]:off[r] + a]) + [pick] + [-1] * (n - a)
    return np.array(acc, np.int32), np.array(tokens, np.int32)


def run_verify(hq, p, q, drafts, off, u, us, stream=None):
    R, V, D = len(off) - 1, p.shape[1], len(drafts)
    acc = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((D + R,), -7, dtype=torch.int32, device="cuda")
    hq.hq_verify_drafts(dev(p), None if q is None else dev(q), dev(drafts) if D else None, dev(off), dev(u) if D else None,
                        dev(us), acc, tokens, R, D, V, stream=stream)
    return acc.cpu().numpy(), tokens.cpu().numpy()


def verify_case(seed, lengths, V, near=0.5):
    g = synthetic.rng(seed)
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    R, D = len(lengths), int(off[-1])
    soft = lambda l: (np.exp(l - l.max(-1, keepdims=True)) / np.exp(l - l.max(-1, keepdims=True)).sum(-1, keepdims=True))
    l = g.standard_normal((D + R, V)) * 2
    p = soft(l).astype(np.float32)
    at = np.arange(D) + np.repeat(np.arange(R), lengths)
    q = soft(l[at] + near * g.standard_normal((D, V))).astype(np.float32) if D else np.zeros((0, V), np.float32)
    drafts = np.array([g.choice(V, p=row.astype(np.float64) / row.astype(np.float64).sum()) for row in q], np.int32)
    return p, q, drafts, off, g.random(D, dtype=np.float32), g.random(R, dtype=np.float32)


@pytest.mark.parametrize("V", [1, 2, 33, 1000, 1024, 4099, 50_001])
@pytest.mark.parametrize("sure", [False, True])
def test_verify(hq, V, sure):
    for seed, lengths in enumerate(([4], [0], [0, 0, 0], [3, 0, 8, 1, 0, 5, 2], [1] * 40)):
        p, q, drafts, off, u, us = verify_case(900 + seed, lengths, V)
        q = None if sure else q
        if sure:
            u = u * 0.2
        got = run_verify(hq, p, q, drafts, off, u, us)
        ref = verify_reference(p, q, drafts, off, u, us)
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]), lengths


def test_verify_edges(hq):
    """Equal distributions (nothing left of the residual), zero rows, NaN, uniform
    numbers at their ends, the first and the last token of the vocabulary."""
    V = 3001
    p, q, drafts, off, u, us = verify_case(950, [2, 2, 2, 2, 2, 2], V)
    at = np.arange(12) + np.repeat(np.arange(6), 2)
    q[0:2] = p[at[0:2]]
    p[at[0], drafts[0]] = 0
    q[0] = p[at[0]]                                    # refused with p == q: the residual is empty
    p[3] = 0                                           # request 1: a zero target row: -1
    p[6, ::7] = np.nan
    q[4, 5::9] = np.nan
    u[6:8], us[3] = 0, np.float32(1) - np.float32(2.0 ** -24)
    us[4] = 0
    p[at[8], :] = 0
    p[at[8], V - 1] = 1
    p[at[10], :] = 0
    p[at[10], 0] = 0.25
    got = run_verify(hq, p, q, drafts, off, u, us)
    ref = verify_reference(p, q, drafts, off, u, us)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    assert -1 in got[1][off[1] + 1:off[1] + 2]


def test_verify_samples_the_distribution(hq):
    """All accepted, the bonus token over 4096 uniform numbers: frequencies within
    the fixed-point quantiles (an exact count, not a statistical one)."""
    V, R = 257, 4096
    g = synthetic.rng(960)
    w = g.random(V).astype(np.float32)
    w[::4] = 0
    row = (w / w.sum()).astype(np.float32)
    p = np.tile(row, (R, 1))
    us = (np.arange(R, dtype=np.float32) + np.float32(0.5)) / np.float32(R)
    off = np.zeros(R + 1, np.int32)
    acc, tokens = run_verify(hq, p, None, np.zeros(0, np.int32), off, np.zeros(0, np.float32), us)
    c = np.cumsum(np.floor(row.astype(np.float64) * 2.0 ** 40))
    assert np.array_equal(tokens, np.searchsorted(c, np.floor(us.astype(np.float64) * c[-1]), side="right"))
    assert (acc == 0).all() and not (tokens % 4 == 0).any()


def test_verify_reports_bad_input(hq):
    V = 100
    p, q, drafts, off, u, us = verify_case(970, [3, 2, 1], V)
    u[:] = 0
    drafts[1] = V
    got = run_verify(hq, p, q, drafts, off, u, us)
    assert hq.hq_device_fault() & 0xFF == hq.HQ_FAULT_DRAFT
    ref = verify_reference(p, q, drafts, off, u, us)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    drafts[1] = -1
    got = run_verify(hq, p, None, drafts, off, u, us)
    assert hq.hq_device_fault() & 0xFF == hq.HQ_FAULT_DRAFT
    ref = verify_reference(p, None, drafts, off, u, us)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
    bad = off.copy()
    bad[1] = 7
    drafts[1] = 3
    acc, tokens = run_verify(hq, p, q, drafts, bad, u, us)
    assert hq.hq_device_fault() & 0xFF == hq.HQ_FAULT_DRAFT
    assert acc[0] == -7 and acc[1] == -7 and acc[2] >= 0
