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
