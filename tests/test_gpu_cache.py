"""GPU tests of the quantized key/value cache: what is written against the blocks' definition (bit by bit), what is read,
and attention against its formula in 64 bits on the stored values.

Tolerance of attention.  With weights p_i of the formula, an error d_i of score i changes the output by at most
2 max|d| sum p|v| (numerator and denominator), and so does a relative error of the weights.
  scores: scale * sum|q k| times: f32: q in two terms 2^-22, sums in fp32 of head_dim / 16 tensor-core steps, the blocks and
          the scales, below 2^-20 together; f16 and bf16: a stored key rounded to 11 bits 2^-11 (or 2^-19 of the largest
          key near it), and the sums.  The argument of the power is a product and a difference in fp32: 2^-23 (|s| + |max|).
  weights: the power 2^-21; f16 and bf16: a rounding to 11 bits of the weight, of the weight times the value's scale, and of the
          stored value, 2^-11 each; f32: two terms, 2^-21.  Weights below 2^-24 of the largest may vanish (their number times
          2^-24 of the largest |v| there; f32, where scales are held in [2^8, 2^9) and the second term is rounded to 2^-25: 2^-33);
          the same for values far below others near them (2^-19 of the largest).
  sums:   n positions in fp32, the accumulators truncating: n / 16 steps of 2^-23 at most, of the sum of |terms|.
The output is rounded once, half a step of its type.
"""
from __future__ import annotations

import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import synthetic

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
BITS = {"q8_0": 8, "q4_0": 4}


@pytest.fixture(scope="module")
def hq():
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    hq.hq_device_fault()
    return hq


@pytest.fixture(autouse=True)
def no_device_fault(hq):
    yield
    assert hq.hq_device_fault() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ the definition

def stored(x, fmt):
    """[..., dim] fp32 -> (scales fp16 [..., dim/32], quants [..., dim], signed) as hq.h defines them."""
    f = np.float32
    w = np.ascontiguousarray(x, f).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        first = np.abs(w).argmax(-1)[..., None]
        m = np.take_along_axis(w, first, -1)
        d = np.minimum(np.abs(m) / f(127), f(65504)) if fmt == "q8_0" else np.clip(m / f(-8), f(-65504), f(65504))
        z = np.where(d == 0, f(0), w / np.where(d == 0, f(1), d)).astype(f)
        if fmt == "q8_0":
            q = np.clip(np.trunc(z.astype(np.float64) + np.copysign(0.5, z)), -127, 127)
        else:
            q = np.where(d == 0, 0, np.clip(np.floor((z + f(8.5)).astype(f)), 0, 15) - 8)
        odd = ~np.isfinite(w).all(-1, keepdims=True)
        d = np.where(odd, f(np.nan), d).astype(np.float16)
        q = np.where(odd, 0, q)
    return d[..., 0], q.reshape(x.shape).astype(np.int64)


def values(d, q):
    with np.errstate(all="ignore"):
        return (q.reshape(*d.shape, 32) * d.astype(np.float64)[..., None]).reshape(q.shape)


def cell_bytes(k, v, fmt):
    """One cell (16 positions of a head) from scales and quants of its keys and values, laid out as hq.h says."""
    (kd, kq), (vd, vq) = k, v
    bits, dim = BITS[fmt], kq.shape[-1]
    lane = dim * bits // 8 // 4
    unit, mid = min(16, lane), 128 if bits == 8 else 8
    out = bytearray()

    def word(e):                                # of 8 elements of a block: its bytes
        e = [int(i) + mid for i in e]
        if bits == 8:
            return bytes(e)
        return sum(e[i] << (4 * (i // 2 + 4 * (i % 2))) for i in range(8)).to_bytes(4, "little")
    for p in range(16):
        lanes = [b"".join(word(kq[p, 32 * b + 8 * c:32 * b + 8 * c + 8]) for b in range(dim // 32)) for c in range(4)]
        for u in range(lane // unit):
            for c in range(4):
                out += lanes[c][u * unit:(u + 1) * unit]
    for p in range(0, 16, 2):
        lanes = []
        for g in range(8):
            s = b""
            for b in range(dim // 32):
                e = [[int(vq[p + h, 32 * b + 8 * j + g]) + mid for j in range(4)] for h in (0, 1)]
                if bits == 8:
                    s += bytes(e[0][:2] + e[1][:2] + e[0][2:] + e[1][2:])
                else:
                    s += sum(n << (4 * j + 16 * h) for h in (0, 1) for j, n in enumerate(e[h])).to_bytes(4, "little")
            lanes.append(s)
        for u in range(lane // unit):
            for g in range(8):
                out += lanes[g][u * unit:(u + 1) * unit]
    out += kd.astype(np.float16).tobytes()
    out += vd.astype(np.float16).reshape(8, 2, -1).transpose(0, 2, 1).tobytes()
    return bytes(out)


# ------------------------------------------------------------------ a batch

class Batch:
    """Requests with `new[r]` tokens and lengths[r] positions, their pages in mixed order in a pool of random bytes."""

    def __init__(self, hq, g, fmt, kv, dim, page, lengths, new, dtype="f32", width=None, tail=3):
        self.hq, self.fmt, self.kv, self.dim, self.page, self.dtype = hq, fmt, kv, dim, page, dtype
        self.lengths, self.new = np.asarray(lengths, np.int32), np.asarray(new, np.int32)
        need = -(-self.lengths // page)
        self.width = width or max(1, int(need.max(initial=0)))
        self.n_pages = int(need.sum()) + 2
        order = g.permutation(self.n_pages).astype(np.int32)
        self.table = g.integers(-9, 1 << 30, (len(lengths), self.width)).astype(np.int32)       # what is behind is not read
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.offsets[-1]) + tail
        self.page_bytes = hq.hq_cache_page_bytes(hq.FMT_CODES[fmt], kv, dim, page)
        self.pool = dev(g.integers(0, 256, self.n_pages * self.page_bytes).astype(np.uint8))
        self.d_table, self.d_offsets, self.d_lengths = dev(self.table), dev(self.offsets), dev(self.lengths)

    def args(self, offsets=None, T=None):
        return (self.pool, self.n_pages, self.page, self.d_table, self.width, self.d_offsets if offsets is None else offsets,
                self.d_lengths, len(self.lengths), self.T if T is None else T)

    def write(self, k, v, offsets=None, stream=None):
        """k, v [T][kv][dim] on the device, of any token stride."""
        hq = self.hq
        code = {t: hq.DTYPE_CODES[n] for n, t in DT.items()}[k.dtype]
        hq.hq_cache_write(hq.FMT_CODES[self.fmt], k, k.stride(0), v, v.stride(0), *self.args(offsets, k.shape[0]), self.kv,
                          self.dim, code, stream=stream)

    def fill(self, g, scale=1.0):
        """Every position of every request written, in one call; returns the values that are then stored, by request."""
        n = int(self.lengths.sum())
        k = (g.standard_normal((n, self.kv, self.dim)) * scale).astype(np.float32)
        v = (g.standard_normal((n, self.kv, self.dim)) * scale).astype(np.float32)
        k *= 1 + 4 * (g.uniform(0, 1, self.dim) < 0.05).astype(np.float32)
        off = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        if n:
            self.write(dev(k), dev(v), dev(off))
        k, v = values(*stored(k, self.fmt)), values(*stored(v, self.fmt))
        return [(k[a:b], v[a:b]) for a, b in zip(off[:-1], off[1:])]

    def read(self, dtype, offsets=None, T=None, fill=None):
        hq, T = self.hq, self.T if T is None else T
        k, v = (torch.full((T, self.kv, self.dim), 77.0 if fill is None else fill, dtype=DT[dtype], device="cuda") for _ in "kv")
        hq.hq_cache_read(hq.FMT_CODES[self.fmt], k, k.stride(0), v, v.stride(0), *self.args(offsets, T), self.kv, self.dim,
                         hq.DTYPE_CODES[dtype])
        return k, v

    def attend(self, q, heads, causal=1, window=0, scale=None, out=None, ws=None, stream=None):
        hq = self.hq
        code = {t: hq.DTYPE_CODES[n] for n, t in DT.items()}[q.dtype]
        if out is None:
            out = torch.full((q.shape[0], heads, self.dim), 77.0, dtype=q.dtype, device="cuda")
        if ws is None:
            n = hq.hq_cache_attention_workspace(hq.FMT_CODES[self.fmt], self.page, self.width, len(self.lengths), q.shape[0],
                                                heads, self.kv, self.dim, code)
            ws = torch.full((max(1, n),), 255, dtype=torch.uint8, device="cuda")
        hq.hq_cache_attention(hq.FMT_CODES[self.fmt], q, q.stride(0), *self.args(T=q.shape[0]), heads, self.kv, self.dim,
                              self.dim ** -0.5 if scale is None else scale, causal, window, out, out.stride(0), code, ws,
                              ws.numel(), stream=stream)
        return out


def formula(q, cache, lengths, new, heads, kv, dim, causal, window, scale):
    """Outputs and the tolerance's parts in 64 bits: out, 2 * (score error factor), see the top of the file."""
    outs, scores, spread, mags, count, big = [], [], [], [], [], []
    at = 0
    for r, n in enumerate(new):
        k, v = (torch.from_numpy(x).cuda() for x in cache[r])
        for i0 in range(0, int(n), 64):
            i1 = min(int(n), i0 + 64)
            qq = q[at + i0:at + i1].double().reshape(i1 - i0, kv, heads // kv, dim)
            L = int(lengths[r])
            pos = L - int(n) + torch.arange(i0, i1, device="cuda")[:, None]
            p = torch.arange(L, device="cuda")[None]
            see = torch.ones((i1 - i0, L), dtype=torch.bool, device="cuda")
            if causal:
                see &= p <= pos
            if window:
                see &= p > pos - window
            if not causal:
                see &= True
            see = see[:, None, None]
            s = torch.einsum("nkgd,lkd->nkgl", qq, k) * scale
            e = torch.einsum("nkgd,lkd->nkgl", qq.abs(), k.abs()) * abs(scale)
            s = s.masked_fill(~see, -float("inf"))
            m = s.amax(-1, keepdim=True) if L else s.sum(-1, keepdim=True)
            w = torch.exp(s - torch.where(m == -float("inf"), 0.0, m))
            w = torch.where(see, w, 0.0)
            z = w.sum(-1, keepdim=True)
            w = w / torch.where(z == 0, 1.0, z)
            vv = torch.where(torch.isfinite(v), v, 0.0)
            outs.append(torch.einsum("nkgl,lkd->nkgd", w, vv).reshape(i1 - i0, heads, dim))
            mags.append(torch.einsum("nkgl,lkd->nkgd", w, vv.abs()).reshape(i1 - i0, heads, dim))
            shape = (i1 - i0, heads, 1)
            zero = torch.zeros(shape, dtype=torch.float64, device="cuda")
            scores.append(torch.where(see, e, 0.0).amax(-1).reshape(shape) if L else zero)
            spread.append(torch.where(see & (w > 1e-12), s.abs(), 0.0).amax(-1).reshape(shape) if L else zero)
            # a term lost below 2^-24 of the largest weight: n of them, of the largest |v|
            lost = (see.double().sum(-1) * w.amax(-1)).reshape(shape) if L else zero
            count.append(lost * (vv.abs().amax() if L else 0.0))
            big.append(zero + (see.double().sum(-1).amax() if L else 0.0))
        at += int(n)
    cat = [torch.cat(x) if x else torch.zeros((0, heads, 1), device="cuda") for x in (outs, mags, scores, spread, count, big)]
    return cat


def check_attention(out, q, cache, lengths, new, heads, kv, dim, dtype, causal=1, window=0, scale=None, what=""):
    scale = dim ** -0.5 if scale is None else scale
    ref, mag, score, spread, lost, seen = formula(q, cache, lengths, new, heads, kv, dim, causal, window, scale)
    n = ref.shape[0]
    got = out[:n].double()
    if dtype == "f32":
        ds, dw, tiny = score * 2.0 ** -20, 2.0 ** -20, 2.0 ** -33
    else:
        ds, dw, tiny = score * (2.0 ** -11 + 2.0 ** -17), 2.0 ** -10, 2.0 ** -24
    ds = ds + spread * 2.0 ** -22
    tol = (2 * torch.expm1(ds) + 2 * dw + (seen / 16 + 16) * 2.0 ** -23) * mag + lost * (tiny + 2.0 ** -20 * ds)
    if dtype != "f32":
        tol = tol + 2.0 ** -19 * mag.amax(-1, keepdim=True)
    tol = tol + HALF_STEP[dtype] * (ref.abs() + tol) + 2.0 ** -25
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - ref).abs()[bad].max()), float(tol[bad].min()),
                                 torch.nonzero(bad)[:3].tolist())


# ------------------------------------------------------------------ rows written and read

LENGTHS = [(1, 1), (16, 16), (17, 5), (0, 0), (33, 33), (129, 2), (40, 0), (64, 31)]


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dim,kv,page", [(64, 3, 16), (128, 1, 64), (128, 8, 32), (256, 2, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_written_rows_read_back(hq, fmt, dim, kv, page, dtype):
    """Rows of a wider matrix, ragged requests: the values of the blocks' definition to the bit, nothing else touched."""
    g = synthetic.rng(1000 + dim + kv + page)
    b = Batch(hq, g, fmt, kv, dim, page, *zip(*LENGTHS), tail=4)
    before = b.pool.clone()
    x = torch.from_numpy(g.standard_normal((b.T, 2 * kv + 1, dim)).astype(np.float32)).cuda()
    x[:, :, 32:40] = 0
    x[3, 0] = 0                                 # blocks of zeros
    x[5, :, :32] = 1.5                          # a block of equal values
    x[6, 0, ::7] *= -1e-6
    x = x.to(DT[dtype])
    k, v = x[:, :kv], x[:, kv + 1:]
    b.write(k, v)
    n = int(b.offsets[-1])
    for out in DT:
        got = b.read(out)
        for rows, y in ((k, got[0]), (v, got[1])):
            want = values(*stored(rows[:n].float().cpu().numpy(), fmt))
            assert torch.equal(y[:n], torch.from_numpy(want).cuda().to(DT[out])), out
            assert bool((y[n:] == 77).all())
    # positions that no token was written to keep their bytes
    cells = b.page // 16
    changed = (b.pool != before).view(b.n_pages, kv, cells, -1).any(-1).any(1).cpu().numpy()
    mine = np.zeros((b.n_pages, cells), bool)
    for r, (length, new) in enumerate(LENGTHS):
        for p in range(length - new, length):
            mine[b.table[r, p // page], p % page // 16] = True
    assert not (changed & ~mine).any()


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layout(hq, fmt, dim):
    """A cell's bytes are those that hq.h describes."""
    g = synthetic.rng(1100 + dim)
    b = Batch(hq, g, fmt, 2, dim, 32, [32], [32], tail=0)
    k, v = (g.standard_normal((32, 2, dim)).astype(np.float32) for _ in "kv")
    b.write(dev(k), dev(v))
    (kd, kq), (vd, vq) = stored(k, fmt), stored(v, fmt)
    want = b"".join(cell_bytes((kd[p:p + 16, h], kq[p:p + 16, h]), (vd[p:p + 16, h], vq[p:p + 16, h]), fmt)
                    for h in (0, 1) for p in (0, 16))
    got = b.pool.view(b.n_pages, -1)[int(b.table[0, 0])].cpu().numpy().tobytes()
    assert got == want


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_values_that_are_no_numbers_and_very_large_ones(hq, fmt):
    g = synthetic.rng(1110)
    b = Batch(hq, g, fmt, 1, 128, 16, [9], [9], tail=0)
    x = g.standard_normal((9, 1, 128)).astype(np.float32)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 127], x[3, 0, 64] = np.nan, np.inf, -np.inf, 3e38
    x[4, 0, :32] *= 1e7
    x[5, 0] *= 1e-9
    x[6, 0, 5] = -3e38
    x[7, 0] = 1e-45
    k = dev(x)
    b.write(k, k.flip(2))
    got = b.read("f32")
    for y, rows in zip(got, (x, x[:, :, ::-1])):
        want = torch.from_numpy(values(*stored(rows, fmt))).float().cuda()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(y, nan=5.0), torch.nan_to_num(want, nan=5.0))
        assert int(torch.isnan(y).sum()) == 3 * 32


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_quotients_are_those_of_a_division(hq, fmt, dtype):
    """Millions of blocks of every size, many of whose quotients lie at the middle between two quants: to the bit."""
    g = synthetic.rng(1115)
    n, dim = 9000, 256
    b = Batch(hq, g, fmt, 1, dim, 256, [n], [n], tail=0)
    x = g.standard_normal((n, 1, dim)).astype(np.float32) * np.exp2(g.integers(-14, 15, (n, 1, 1))).astype(np.float32)
    if dtype == "f32":
        x[::3] *= np.exp2(g.integers(-110, 90, (len(x[::3]), 1, 1))).astype(np.float32)
    top = np.abs(x.reshape(n, 1, -1, 32)).max(-1, keepdims=True)
    half = top * (g.integers(-253, 254, (n, 1, dim // 32, 32)) / (254 if fmt == "q8_0" else 16)).astype(np.float32)
    x = np.where(g.uniform(0, 1, (n, 1, dim // 32, 32)) < 0.5, x.reshape(n, 1, -1, 32), np.clip(half, -top, top)).reshape(n, 1, dim)
    k = dev(x).to(DT[dtype])
    k = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    b.write(k, k.flip(2))
    got = b.read("f32")
    for y, rows in zip(got, (k, k.flip(2))):
        want = values(*stored(rows.float().cpu().numpy(), fmt))
        assert torch.equal(y, torch.from_numpy(want).float().cuda())


def test_tokens_without_a_place_and_pages_out_of_range(hq):
    """A length below the tokens leaves the first ones without a position; a page number out of range reads as NaN."""
    g = synthetic.rng(1120)
    b = Batch(hq, g, "q8_0", 2, 64, 16, [3, 40], [7, 40], tail=1)
    x = torch.from_numpy(g.standard_normal((b.T, 2, 64)).astype(np.float32)).cuda()
    b.write(x, x)
    assert hq.hq_device_fault() == 0
    want = torch.from_numpy(values(*stored(x.cpu().numpy(), "q8_0"))).float().cuda()
    for y in b.read("f32"):
        assert bool((y[:4] == 0).all()) and torch.equal(y[4:47], want[4:47]) and bool((y[47:] == 77).all())
    before = b.pool.clone()
    for bad in (-1, b.n_pages, 2 ** 31 - 1, -2 ** 31):
        b.d_table[1, 1] = bad
        b.write(x + 1, x + 1)
        assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
        for y in b.read("f32"):
            assert bool(torch.isnan(y[7 + 16:7 + 32]).all()) and not bool(torch.isnan(y[:7 + 16]).any())
        assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    b.pool.copy_(before)


@pytest.mark.parametrize("offsets,lengths", [([0, 5, 3, 8], None), ([-1, 5, 6, 8], None), ([0, 2, 5, 99], None),
                                             (None, [5, -1, 20]), (None, [5, 1000, 20])])
def test_descriptors_out_of_range(hq, offsets, lengths):
    """The request is left out and reported; the others' results are their own."""
    g = synthetic.rng(1130)
    b = Batch(hq, g, "q4_0", 1, 128, 16, [5, 9, 20], [2, 3, 3], tail=2)
    cache = b.fill(g)
    x = torch.from_numpy(g.standard_normal((b.T, 4, 128)).astype(np.float32)).cuda().bfloat16()
    if offsets is not None:
        b.d_offsets = dev(np.asarray(offsets, np.int32))
    if lengths is not None:
        b.d_lengths = dev(np.asarray(lengths, np.int32))
    out = b.attend(x, 4)
    assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    b.read("f32")
    assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    b.write(x[:, :1], x[:, 1:2])
    assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
    o = b.offsets if offsets is None else np.asarray(offsets)
    ok = [r for r in range(3) if 0 <= o[r] <= o[r + 1] <= b.T and (lengths is None or 0 <= lengths[r] <= b.width * 16)]
    for r in ok:
        if offsets is None or offsets[:2] == [0, 2]:
            rows = slice(int(o[r]), int(o[r + 1]))
            check_attention(out[rows], x[rows], [cache[r]], [b.lengths[r]], [o[r + 1] - o[r]], 4, 1, 128, "bf16", what=r)
    if lengths is not None:
        assert bool((out[2:5] == 77).all())


# ------------------------------------------------------------------ attention

RAGGED = [(1, 1), (2, 1), (15, 1), (0, 0), (16, 1), (17, 1), (31, 1), (127, 1), (128, 1), (129, 1), (300, 0), (1000, 1)]
DRAFTS = [(1, 1), (5, 5), (16, 3), (17, 8), (0, 0), (130, 5), (64, 2), (257, 7), (700, 4)]
PROMPTS = [(40, 40), (7, 7), (300, 300), (517, 130), (1, 1), (0, 0), (129, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (5, 5, 64, 64), (12, 2, 128, 32), (32, 1, 256, 128), (7, 1, 64, 16),
                                               (48, 3, 128, 256)])
@pytest.mark.parametrize("batch", ["ragged", "drafts", "prompts"])
def test_attention(hq, batch, heads, kv, dim, page, fmt, dtype):
    lengths, new = zip(*{"ragged": RAGGED, "drafts": DRAFTS, "prompts": PROMPTS}[batch])
    g = synthetic.rng(1200 + heads + dim)
    b = Batch(hq, g, fmt, kv, dim, page, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, heads, dim)).astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, heads)
    n = int(b.offsets[-1])
    assert bool((out[n:] == 77).all())
    check_attention(out, q, cache, lengths, new, heads, kv, dim, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal,window", [(0, 0), (1, 1), (1, 7), (1, 64), (1, 130), (1, 10 ** 9)])
@pytest.mark.parametrize("batch", ["ragged", "drafts", "prompts"])
def test_masks(hq, batch, causal, window, dtype):
    lengths, new = zip(*{"ragged": RAGGED, "drafts": DRAFTS, "prompts": PROMPTS}[batch])
    g = synthetic.rng(1300 + window % 1000)
    b = Batch(hq, g, "q8_0", 2, 128, 16, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, 6, 128)).astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, 6, causal, window)
    check_attention(out, q, cache, lengths, new, 6, 2, 128, dtype, causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths,new", [([20000], [1]), ([9000, 1, 12000], [5, 1, 8]), ([4100], [1030]), ([30000], [16])])
def test_long_requests_are_split(hq, lengths, new, dtype):
    g = synthetic.rng(1400)
    b = Batch(hq, g, "q4_0", 2, 128, 64, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, 8, 128)).astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, 8)
    check_attention(out, q, cache, lengths, new, 8, 2, 128, dtype)
    again = b.attend(q, 8)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [3, 40])
def test_rows_past_the_largest_float_are_nan(hq, new, dtype):
    """The largest scale: a row of q that times it is past fp32 is NaN (2^160, times keys of about 1), the others are as ever."""
    g = synthetic.rng(1590 + new)
    b = Batch(hq, g, "q4_0", 2, 64, 16, [70], [new])
    cache = b.fill(g)
    x = g.standard_normal((b.T, 8, 64)) * 2.0 ** -100
    x[1, 2] = 2.0 ** 60
    q = torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, 8, scale=2.0 ** 100)
    assert bool(torch.isnan(out[1, 2]).all())
    q[1, 2], out[1, 2] = 0, b.attend(torch.zeros_like(q), 8, scale=2.0 ** 100)[1, 2]
    check_attention(out, q, cache, [70], [new], 8, 2, 64, dtype, scale=2.0 ** 100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch", ["ragged", "drafts", "prompts"])
def test_scales_signs_and_sizes(hq, batch, dtype):
    """Large scores (a softmax of one position), equal ones, negative and zero scales, caches of very small and large values,
    values that grow from page to page."""
    lengths, new = zip(*{"ragged": RAGGED, "drafts": DRAFTS, "prompts": PROMPTS}[batch])
    for i, (size, scale, qs) in enumerate([(1.0, 3.0, 1.0), (1.0, -0.1, 1.0), (1.0, 0.0, 1.0), (1e-5, 1e4, 1.0), (2e5, 1e-7, 1.0),
                                           (1.0, 1e-30, 1e29), (1.0, 1e20, 1e-21)]):
        g = synthetic.rng(1500 + i)
        b = Batch(hq, g, "q8_0", 2, 64, 16, lengths, new)
        cache = b.fill(g, size)
        q = torch.from_numpy((g.standard_normal((b.T, 8, 64)) * qs).astype(np.float32)).cuda().to(DT[dtype])
        out = b.attend(q, 8, scale=scale)
        check_attention(out, q, cache, lengths, new, 8, 2, 64, dtype, scale=scale, what=(size, scale))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,new", [(4, 1), (4, 3), (8, 40)])
def test_nothing_unseen_touches_a_row(hq, heads, new, dtype):
    """Infinities and NaN in positions that a token does not see (later ones, those before its window, the rest of a page)
    leave its bits alone; in a value it sees they take that block of 32, in a key all of the row."""
    g = synthetic.rng(1600 + new)
    L, at = 200, 200 - new
    b = Batch(hq, g, "q8_0", 1, 128, 16, [L], [new], tail=0)
    k, v = (g.standard_normal((L, 1, 128)).astype(np.float32) for _ in "kv")
    off = dev(np.array([0, L], np.int32))
    q = torch.from_numpy(g.standard_normal((new, heads, 128)).astype(np.float32)).cuda().to(DT[dtype])
    window = 90
    b.write(dev(k), dev(v), off)
    clean = b.attend(q, heads, window=window)
    k2, v2 = k.copy(), v.copy()
    k2[:at - window], v2[:at - window] = np.nan, np.inf         # before every window
    if new > 1:
        k2[-1], v2[-1] = np.inf, np.nan                         # the last token's: only that token sees it
    b.write(dev(k2), dev(v2), off)
    out = b.attend(q, heads, window=window)
    same = new - 1 if new > 1 else 1
    assert torch.equal(out[:same], clean[:same])
    if new > 1:
        assert bool(torch.isnan(out[-1]).all())
    v3 = v.copy()
    v3[L - 2, 0, 40] = np.nan                                   # a value of the token before the last
    b.write(dev(k), dev(v3), off)
    out = b.attend(q, heads, window=window)
    for i in range(new):
        sees = at + i >= L - 2
        assert bool(torch.isnan(out[i, :, 32:64]).all()) == sees
        rest = torch.cat([out[i, :, :32], out[i, :, 64:]], -1)
        want = torch.cat([clean[i, :, :32], clean[i, :, 64:]], -1)
        assert torch.equal(rest, want)
        if not sees:
            assert torch.equal(out[i], clean[i])
    k3 = k.copy()
    k3[L - 2, 0, 3] = -np.inf
    b.write(dev(k3), dev(v), off)
    out = b.attend(q, heads, window=window)
    for i in range(new):
        if at + i >= L - 2:
            assert bool(torch.isnan(out[i]).all())
        else:
            assert torch.equal(out[i], clean[i])
    # a query that is no number keeps to its own row
    q2 = q.clone()
    q2[0, 1, 5] = float("nan")
    b.write(dev(k), dev(v), off)
    out = b.attend(q2, heads, window=window)
    assert bool(torch.isnan(out[0, 1]).all())
    out[0, 1] = clean[0, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,new", [(2, 6), (8, 30)])
def test_rows_that_see_nothing(hq, heads, new, dtype):
    """Tokens at negative positions, and an empty cache that is not causal: zeros."""
    g = synthetic.rng(1700)
    b = Batch(hq, g, "q4_0", 2, 64, 16, [4, 0, 9], [new, 3, 1])
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, heads, 64)).astype(np.float32)).cuda().to(DT[dtype])
    for causal in (1, 0):
        out = b.attend(q, heads, causal)
        if causal:
            assert bool((out[:new - 4] == 0).all())
        assert bool((out[new:new + 3] == 0).all())
        check_attention(out, q, cache, b.lengths, b.new, heads, 2, 64, dtype, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing_whatever_their_query(hq, dtype):
    g = synthetic.rng(1705)
    b = Batch(hq, g, "q8_0", 1, 64, 16, [3, 2], [30, 2])
    b.fill(g)
    q = torch.full((b.T, 8, 64), float("nan"), dtype=DT[dtype], device="cuda")
    out = b.attend(q, 8)
    assert bool((out[:27] == 0).all()) and bool(torch.isnan(out[27:32]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,kv,dim", [(300, 1, 64), (258, 2, 128), (130, 1, 256)])
def test_groups_wider_than_a_tile(hq, heads, kv, dim, dtype):
    """One token's heads in several tiles, the last of them not full."""
    lengths, new = [70, 1, 300, 0], [1, 1, 3, 0]
    g = synthetic.rng(1706 + heads)
    b = Batch(hq, g, "q4_0", kv, dim, 32, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, heads, dim)).astype(np.float32)).cuda().to(DT[dtype])
    out = b.attend(q, heads)
    check_attention(out, q, cache, lengths, new, heads, kv, dim, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_units_of_many_requests_and_windows(hq, dtype):
    """Windows and tokens that do not divide a unit: every block finds its units alike."""
    g = synthetic.rng(1707)
    lengths, new = [1000, 37, 640, 641, 1500, 64], [333, 37, 64, 65, 1, 63]
    b = Batch(hq, g, "q8_0", 3, 64, 64, lengths, new)
    cache = b.fill(g)
    for heads, window in ((9, 0), (15, 63), (21, 65), (3, 200)):
        q = torch.from_numpy(g.standard_normal((b.T, heads, 64)).astype(np.float32)).cuda().to(DT[dtype])
        out = b.attend(q, heads, window=window)
        check_attention(out, q, cache, lengths, new, heads, 3, 64, dtype, 1, window, what=(heads, window))


@pytest.mark.parametrize("heads,new", [(4, 1), (8, 20)])
def test_pages_out_of_range_make_their_rows_nan(hq, heads, new):
    g = synthetic.rng(1710)
    b = Batch(hq, g, "q4_0", 1, 128, 16, [100, 70], [new, new], tail=0)
    b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, heads, 128)).astype(np.float32)).cuda().bfloat16()
    clean = b.attend(q, heads)
    for bad in (-5, b.n_pages, 2 ** 31 - 1):
        b.d_table[0, 2] = bad
        out = b.attend(q, heads)
        assert hq.hq_device_fault() == hq.HQ_FAULT_CACHE
        assert bool(torch.isnan(out[:new]).all()) and torch.equal(out[new:], clean[new:])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("heads,new", [(4, 2), (16, 9)])
def test_rows_of_a_wider_matrix_and_in_place(hq, heads, new, dtype):
    g = synthetic.rng(1720)
    b = Batch(hq, g, "q8_0", 2, 64, 16, [50, 90], [new, new])
    b.fill(g)
    wide = torch.from_numpy(g.standard_normal((b.T, heads + 5, 64)).astype(np.float32)).cuda().to(DT[dtype])
    q = wide[:, 2:2 + heads]
    want = b.attend(q.contiguous(), heads)
    kept = wide.clone()
    out = b.attend(q, heads, out=q)
    n = 2 * new
    assert torch.equal(out[:n], want[:n])
    kept[:n, 2:2 + heads] = want[:n]
    assert torch.equal(wide, kept)


def test_a_pool_past_4_gb(hq):
    """Pages whose bytes lie behind 2^32, and page numbers times heads past 2^31 in all."""
    g = synthetic.rng(1730)
    kv, dim, page = 8, 128, 64
    hqp = hq.hq_cache_page_bytes(8, kv, dim, page)
    n_pages = (5 << 30) // hqp
    b = Batch(hq, g, "q8_0", kv, dim, page, [150, 64, 3], [2, 2, 2], "bf16")
    small = b.pool
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, 16, dim)).astype(np.float32)).cuda().bfloat16()
    want = b.attend(q, 16)
    b.pool = torch.empty(n_pages * hqp, dtype=torch.uint8, device="cuda")
    far = n_pages - small.numel() // hqp
    b.pool.view(n_pages, hqp)[far:] = small.view(-1, hqp)
    b.n_pages, b.d_table = n_pages, b.d_table + far
    assert torch.equal(b.attend(q, 16)[:6], want[:6])
    k, v = b.read("f32")
    for r, first in enumerate(b.offsets[:-1]):
        assert torch.equal(k[first:first + 2].double(), torch.from_numpy(cache[r][0][-2:]).cuda())
    x = torch.ones((b.T, kv, dim), device="cuda")
    b.write(x, x)
    assert bool((b.read("f32")[1][:6] == 127 * np.float16(np.float32(1) / np.float32(127)).astype(np.float64)).all())


def test_in_a_graph_with_other_lengths(hq):
    """Write and attend, captured once and replayed with other rows, lengths and pages: the bits of plain calls."""
    g = synthetic.rng(1740)
    heads, kv, dim = 8, 2, 128
    b = Batch(hq, g, "q4_0", kv, dim, 16, [300, 40, 800], [3, 1, 2], width=64, tail=0)
    whole = Batch(hq, g, "q4_0", kv, dim, 16, [b.n_pages * 16], [0])
    whole.pool, whole.n_pages, whole.d_table = b.pool, b.n_pages, torch.arange(b.n_pages, dtype=torch.int32, device="cuda")[None]
    whole.fill(g)                               # every page of the pool holds numbers
    x = torch.from_numpy(g.standard_normal((b.T, heads + 2 * kv, dim)).astype(np.float32)).cuda().bfloat16()
    n = hq.hq_cache_attention_workspace(4, 16, 64, 3, b.T, heads, kv, dim, 2)
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    out = torch.empty((b.T, heads, dim), dtype=torch.bfloat16, device="cuda")

    def step():
        b.write(x[:, heads:heads + kv], x[:, heads + kv:])
        b.attend(x[:, :heads], heads, out=out, ws=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lengths in ([300, 40, 800], [17, 200, 12], [3, 1, 1000]):
        b.d_lengths.copy_(dev(np.asarray(lengths, np.int32)))
        b.d_table.copy_(dev(g.permutation(b.n_pages)[np.arange(3 * 64) % b.n_pages].reshape(3, 64).astype(np.int32)))
        x.copy_(torch.from_numpy(g.standard_normal(tuple(x.shape)).astype(np.float32)))
        pool = b.pool.clone()
        step()
        want = out.clone(), b.pool.clone()
        assert not bool(torch.isnan(out).any())
        b.pool.copy_(pool)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(b.pool, want[1])


def test_streams_and_two_calls_at_once(hq):
    g = synthetic.rng(1750)
    b = [Batch(hq, g, f, 2, 64, 16, [2000, 30], [1, 4], tail=0) for f in ("q8_0", "q4_0")]
    for i in b:
        i.fill(g)
    q = [torch.from_numpy(g.standard_normal((5, 4, 64)).astype(np.float32)).cuda() for _ in b]
    want = [i.attend(j, 4) for i, j in zip(b, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    outs = [[torch.empty_like(j) for _ in range(8)] for j in q]
    spaces = [torch.empty(max(1, hq.hq_cache_attention_workspace(8, 16, i.width, 2, 5, 4, 2, 64, 0)), dtype=torch.uint8,
                          device="cuda") for i in b]
    torch.cuda.synchronize()
    for n in range(8):
        for i, j, s, o, w in zip(b, q, streams, outs, spaces):
            i.attend(j, 4, out=o[n], ws=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(i, w) for i in o)


def test_many_requests(hq):
    """More requests than a block looks at in one go, most of them without a token."""
    g = synthetic.rng(1760)
    R = 2500
    new = (g.uniform(0, 1, R) < 0.1).astype(np.int32) * g.integers(1, 3, R).astype(np.int32)
    lengths = np.maximum(new, g.integers(0, 40, R)).astype(np.int32)
    b = Batch(hq, g, "q8_0", 1, 64, 16, lengths, new)
    cache = b.fill(g)
    q = torch.from_numpy(g.standard_normal((b.T, 2, 64)).astype(np.float32)).cuda().bfloat16()
    out = b.attend(q, 2)
    check_attention(out, q, cache, lengths, new, 2, 1, 64, "bf16")
    k, v = b.read("f32")
    at = np.repeat(np.arange(R), new)
    for t in range(0, int(b.offsets[-1]), 17):
        r = at[t]
        p = lengths[r] - new[r] + t - b.offsets[r]
        assert torch.equal(k[t].double(), torch.from_numpy(cache[r][0][p]).cuda())
