"""GPU tests of the key/value cache at the ends of what its calls allow.  Tolerances: test_gpu_cache."""
from __future__ import annotations

import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import synthetic
from test_gpu_cache import DT, Batch, check_attention, dev, hq, no_device_fault  # noqa: F401

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
