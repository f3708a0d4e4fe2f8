"""Every kind of bounded wait gives up within its limit and says so, whatever the
fault word holds already (the limit is short, nothing faults or hangs)."""
import time

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def hq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_weight_matvec_hq_gb300 import build
    build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    return hq


@pytest.mark.parametrize("wait", ["HQ_WAIT_MATVEC", "HQ_WAIT_CLUSTER", "HQ_WAIT_MATMUL", "HQ_WAIT_MATMUL_GO"])
@pytest.mark.parametrize("prior", ["", "HQ_FAULT_EXPERT_ID", "HQ_FAULT_ADAPTER_ID", "HQ_FAULT_DRAFT"])
def test_time_out_joins_the_fault_word(hq, wait, prior):
    assert hq.hq_device_fault() == 0
    before = getattr(hq, prior) if prior else 0
    t = time.perf_counter()
    hq.hq_selftest_wait(getattr(hq, wait), before, 2_000_000)          # about a millisecond of SM cycles
    word = hq.hq_device_fault()
    assert time.perf_counter() - t < 1
    assert word & 0xFF == before | hq.HQ_FAULT_WAIT_TIMEOUT
    assert word >> 9 == 0                                               # CTA 0
    assert hq.hq_device_fault() == 0


def test_time_out_takes_its_limit(hq):
    """A wait lasts as long as its limit in SM cycles, not a number of tries."""
    for wait in range(4):
        hq.hq_selftest_wait(wait, 0, 1000)
        hq.hq_device_fault()
        took = []
        for cycles in (2_000_000, 40_000_000):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            hq.hq_selftest_wait(wait, 0, cycles)
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b))
            assert hq.hq_device_fault() & hq.HQ_FAULT_WAIT_TIMEOUT      # (cleared: a wait ends at once while it is set)
        # at 0.5 to 2.5 GHz, and a sleep or so more
        for ms, cycles in zip(took, (2_000_000, 40_000_000)):
            assert cycles / 2.5e6 <= ms <= cycles / 0.5e6 + 20, (wait, took)
