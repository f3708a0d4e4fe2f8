"""GPU tests of the key/value cache at the ends of what its calls allow.  Tolerances: test_gpu_cache."""
from __future__ import annotations

import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import synthetic
from test_gpu_cache import DT, Batch, check_attention, dev, formula, hq, no_device_fault, stored, values  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype,new", [("bf16", 40), ("f16", 3), ("f32", 3)])
def test_rows_written_by_the_call_in_front(hq, dtype, new):
    """Written and attended to without a pause, over places that the attention before has just read: the bits of calls that
    wait for one another."""
    g = synthetic.rng(1770)
    heads, kv, dim = 8, 2, 128
    b = Batch(hq, g, "q8_0", kv, dim, 16, [700] * 8, [new] * 8, tail=0)
    b.fill(g)
    x = [torch.from_numpy(g.standard_normal((b.T, heads + 2 * kv, dim)).astype(np.float32)).cuda().to(DT[dtype]) for _ in range(6)]

    def step(i):
        b.write(x[i][:, heads:heads + kv], x[i][:, heads + kv:])
        return b.attend(x[i][:, :heads], heads, ws=ws, out=outs[i])
    n = hq.hq_cache_attention_workspace(8, 16, b.width, 8, b.T, heads, kv, dim, hq.DTYPE_CODES[dtype])
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((b.T, heads, dim), dtype=DT[dtype], device="cuda") for _ in x]
    want = []
    for i in range(len(x)):
        b.write(x[i][:, heads:heads + kv], x[i][:, heads + kv:])
        torch.cuda.synchronize()
        want.append(b.attend(x[i][:, :heads], heads, ws=ws, out=outs[i]).clone())
        torch.cuda.synchronize()
    for _ in range(20):
        for i in range(len(x)):
            step(i)
        assert all(torch.equal(a, w) for a, w in zip(outs, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,new", [([40, 7, 300, 517, 1, 0, 129], [40, 7, 300, 130, 1, 0, 128]), ([16, 130, 64], [3, 5, 2])])
def test_windows_of_any_size(hq, lengths, new, dtype):
    """A window past every position is no window, to the bit: up to the largest number that the call takes."""
    g = synthetic.rng(1780)
    b = Batch(hq, g, "q8_0", 2, 128, 16, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, 6, 128)).astype(np.float32)).cuda().to(DT[dtype])
    want = b.attend(q, 6)
    check_attention(want, q, cache, lengths, new, 6, 2, 128, dtype)
    for window in (b.width * 16, 2 ** 30, 2 ** 31 - 1, 2 ** 31 + 7, 2 ** 40, 2 ** 63 - 20, 2 ** 63 - 1):
        assert torch.equal(b.attend(q, 6, window=window), want), window
    below = b.attend(q, 6, window=b.width * 16 - 1)             # (hides nothing either, but is counted as a window)
    check_attention(below, q, cache, lengths, new, 6, 2, 128, dtype)


@pytest.mark.parametrize("R,spoil", [(3, {2: -1}), (3, {1: 1 << 30}), (3, {0: -5}), (64, {33: -1}), (64, {20: -(2 ** 31)}), (64, {40: 2 ** 31 - 1}),
                                     (64, {3: 10 ** 6, 31: -7, 32: -7, 60: -1}), (700, {k: -1 for k in range(0, 700, 50)}), (64, {64: 10 ** 6}),
                                     (1, {0: -1})])
def test_a_bad_offset_leaves_out_its_own_requests_alone(hq, R, spoil):
    """Wherever offsets are out of range: the rows of every good request are written and read, and no others."""
    g = synthetic.rng(1790 + R)
    new = g.integers(0, 4, R).astype(np.int32)
    new[0] = 3
    lengths = new + g.integers(0, 30, R).astype(np.int32)
    b = Batch(hq, g, "q8_0", 2, 64, 16, lengths, new, tail=5)
    start = b.pool.clone()
    o = b.offsets.copy()
    for i, x in spoil.items():
        o[i] = x
    good = [r for r in range(R) if 0 <= o[r] <= o[r + 1] <= b.T]
    x = torch.from_numpy(g.standard_normal((b.T, 2, 64)).astype(np.float32)).cuda()
    want_k = torch.full_like(x, 77.0)
    want_v = want_k.clone()
    table, whole = b.d_table, (b.d_offsets, b.d_lengths, b.lengths)
    for r in good:                              # each in a call of its own
        b.d_table, b.d_lengths, b.lengths = table[r:r + 1], dev(lengths[r:r + 1]), lengths[r:r + 1]
        off = dev(o[r:r + 2])
        b.write(x, -x, off)
        hq.hq_cache_read(8, want_k, want_k.stride(0), want_v, want_v.stride(0), *b.args(off), 2, 64, 0)
    assert hq.hq_device_fault() == 0
    want = b.pool.clone()
    b.d_table, (_, b.d_lengths, b.lengths) = table, whole
    b.pool.copy_(start)
    off = dev(o)
    b.write(x, -x, off)
    assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    assert torch.equal(b.pool, want)
    k, v = b.read("f32", off)
    assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_in_front_of_the_first_request(hq, dtype):
    """Offsets need not begin at 0: the rows in front are no request's."""
    g = synthetic.rng(1795)
    b = Batch(hq, g, "q4_0", 2, 64, 16, [9, 30], [4, 2], tail=0)
    cache = b.fill(g)
    b.d_offsets, b.T = b.d_offsets + 6, b.T + 8
    q = torch.from_numpy(g.standard_normal((b.T, 4, 64)).astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, 4)
    for rows in (out, *b.read("f32")):
        assert bool((rows[:6] == 77).all()) and bool((rows[12:] == 77).all()) and not bool((rows[6:12] == 77).any())
    check_attention(out[6:], q[6:], cache, [9, 30], [4, 2], 4, 2, 64, dtype)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype,heads,new", [("bf16", 4, 2), ("f16", 8, 2), ("f32", 16, 3), ("bf16", 16, 9), ("f16", 8, 40)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_scales(hq, fmt, dtype, heads, new, dim):
    """A pool from elsewhere: an infinite scale of a key makes the rows that see it NaN, whatever sign their sums with its quants
    have; that of a value its block of 32.  Other rows keep their bits."""
    g = synthetic.rng(1850 + dim + heads)
    L = 150
    b = Batch(hq, g, fmt, 1, dim, 32, [L], [new], tail=0)
    b.fill(g)
    q = torch.from_numpy(g.standard_normal((new, heads, dim)).astype(np.float32)).cuda().to(DT[dtype])
    clean = {scale: b.attend(q, heads, scale=scale) for scale in (0.1, -0.1)}
    bits, nb = {"q8_0": 8, "q4_0": 4}[fmt], dim // 32
    quants = 2 * 16 * dim * bits // 8
    cell = quants + 2 * 16 * nb * 2
    pool = b.pool.view(torch.int16)
    for p, block in ((3, 0), (L - 2, nb - 1), (L - 1, 1)):
        at = int(b.table[0, p // 32]) * b.page_bytes + p % 32 // 16 * cell + quants
        key = at + (p % 16 * nb + block) * 2
        value = at + 16 * nb * 2 + ((p % 16 // 2 * nb + block) * 2 + p % 2) * 2
        sees = torch.arange(L - new, L, device="cuda") >= p
        for where in (key, value):
            kept = pool[where // 2].clone()
            for infinity in (0x7c00, 0xfc00 - 0x10000):
                pool[where // 2] = infinity
                for scale in clean:
                    out = b.attend(q, heads, scale=scale)
                    want = clean[scale].clone()
                    if where == key:
                        want[sees] = float("nan")
                    else:
                        want[sees, :, 32 * block:32 * block + 32] = float("nan")
                    assert torch.equal(torch.isnan(out), torch.isnan(want)), (p, where == key, infinity, scale)
                    assert torch.equal(out[~torch.isnan(want)], want[~torch.isnan(want)])
            pool[where // 2] = kept


@pytest.mark.parametrize("fmt,bound", [("q4_0", 2.0 ** -17), ("q8_0", 2.0 ** -20)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_far_below_others_in_tiles(hq, fmt, bound, dim):
    """Rows that see one position each give its stored values: 11 bits, or `bound` of the largest that the scales of 32
    neighbouring positions allow (test_tile_rounding has the proof), times a weight over itself (2^-11: the weight's own 11 bits,
    the power and the quotient), rounded to f16."""
    g = synthetic.rng(1900 + dim)
    n, heads = 256, 2
    b = Batch(hq, g, fmt, 1, dim, 64, [n], [n], "f16", tail=0)
    size = np.exp2(-g.uniform(0, 13, (n, 1, dim // 32, 1)))
    size[::8] = 1                               # the largest is near every position
    v = (g.uniform(-1, 1, (n, 1, dim // 32, 32)) * size * 512).astype(np.float32).reshape(n, 1, dim)
    b.write(torch.zeros((n, 1, dim), device="cuda"), dev(v))
    d, quants = stored(v, fmt)
    exact = torch.from_numpy(values(d, quants)).cuda()
    most = np.abs(d.astype(np.float64)).reshape(n // 32, -1).max(1).repeat(32) * (127 if fmt == "q8_0" else 8)
    q = torch.zeros((n, heads, dim), dtype=torch.float16, device="cuda")
    got = b.attend(q, heads, window=1).double()
    tol = bound * torch.from_numpy(most).cuda()[:, None, None] + 2.0 ** -10 * exact.abs()
    tol = tol + 2.0 ** -11 * (exact.abs() + tol) + 2.0 ** -25
    assert bool(((got - exact).abs() <= tol).all()), float(((got - exact).abs() / tol).max())


@pytest.mark.parametrize("dtype,heads,new", [("bf16", 2, 6), ("f32", 2, 6), ("f16", 8, 30)])
def test_tokens_at_negative_positions(hq, dtype, heads, new):
    """Causal: zeros.  Not causal: what their request's other tokens see, to the bit with the same query."""
    g = synthetic.rng(1950)
    b = Batch(hq, g, "q8_0", 1, 64, 16, [4, 1], [new, 3])
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((1, heads, 64)).astype(np.float32)).cuda().to(DT[dtype]).repeat(b.T, 1, 1)
    out = b.attend(q, heads, causal=1)
    assert bool((out[:new - 4] == 0).all()) and bool((out[new:new + 2] == 0).all())
    check_attention(out, q, cache, [4, 1], [new, 3], heads, 1, 64, dtype)
    out = b.attend(q, heads, causal=0)
    for rows in (out[:new], out[new:new + 3]):
        assert torch.equal(rows, rows[-1:].expand_as(rows)) and bool((rows != 0).any())
    check_attention(out, q, cache, [4, 1], [new, 3], heads, 1, 64, dtype, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [2, 40])
def test_one_request_in_different_batches(hq, dtype, new):
    """Alone, beside requests without tokens and before rows that are no request's: either kernel runs, by the mean request.  The
    bits may differ between these, each is within the tolerance, and the same call gives the same bits."""
    g = synthetic.rng(1960 + new)
    heads, kv, dim, L = 8, 2, 128, 333
    q = torch.from_numpy(g.standard_normal((new + 200, heads, dim)).astype(np.float32)).cuda().to(DT[dtype])
    for idle in (0, 1, 15, 63):
        for tail in (0, 200):
            g = synthetic.rng(1961)
            b = Batch(hq, g, "q4_0", kv, dim, 16, [L] + [50] * idle, [new] + [0] * idle, tail=tail)
            cache = b.fill(g)
            rows = q[:new + tail]
            out = b.attend(rows, heads)
            assert bool((out[new:] == 77).all())
            check_attention(out, rows, cache, [L], [new], heads, kv, dim, dtype, what=(idle, tail))
            assert torch.equal(b.attend(rows, heads), out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 256])
def test_one_workspace_for_batches_of_every_size(hq, dim, dtype):
    """What 64 single tokens need is enough for each batch of fewer tokens or requests; nothing behind it is written."""
    g = synthetic.rng(1970 + dim)
    heads, kv = 8, 2
    need = hq.hq_cache_attention_workspace(8, 16, 64, 64, 64, heads, kv, dim, hq.DTYPE_CODES[dtype])
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    for lengths, new in (([300] * 64, [1] * 64), ([900], [64]), ([900], [1]), ([700, 800], [5, 30]), ([90] * 20, [3] * 20)):
        b = Batch(hq, g, "q8_0", kv, dim, 16, lengths, new, width=64, tail=0)
        b.fill(g)
        q = torch.from_numpy(g.standard_normal((b.T, heads, dim)).astype(np.float32)).cuda().to(DT[dtype])
        assert torch.equal(b.attend(q, heads, ws=ws[:need]), b.attend(q, heads))
        assert bool((ws[need:] == 255).all())


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [2, 200])
def test_f16_outputs_are_near_their_own_rounding(hq, fmt, dim, new):
    """Over many outputs, f16 rows are off by at most 1.5 times what rounding the formula's results to f16 is.  Beside that rounding, either
    kernel rounds one more number of 11 bits for every term of an output (a weight, or a weight times a scale), whose error over
    many terms of random sign is no larger, relative to the result: sqrt(2) in all, and the rest of the errors is 2^-3 of it."""
    g = synthetic.rng(1980 + dim)
    heads, kv, L = 8, 2, 3000
    b = Batch(hq, g, fmt, kv, dim, 64, [L], [new], "f16", tail=0)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((new, heads, dim)).astype(np.float32)).cuda().half()
    out = b.attend(q, heads).double()
    ref = formula(q, cache, [L], [new], heads, kv, dim, 1, 0, dim ** -0.5)[0]
    off, rounding = (out - ref).norm() / ref.norm(), (ref.half().double() - ref).norm() / ref.norm()
    assert off <= 1.5 * rounding, (float(off), float(rounding))
