"""Refusals of the wait self-test, checked on the host before a device is touched."""
import pytest

from quantized_weight_matvec_hq_gb300 import build as hq_build


@pytest.fixture(scope="module")
def hq():
    hq_build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    return hq


def test_wait_selftest_refusals(hq):
    L = hq.lib()
    assert L.hq_selftest_wait(-1, 0, 1000, 0) == L.hq_selftest_wait(4, 0, 1000, 0) == hq.HQ_ERR_UNSUPPORTED
    assert L.hq_selftest_wait(0, hq.HQ_FAULT_WAIT_TIMEOUT, 1000, 0) == hq.HQ_ERR_UNSUPPORTED
    assert L.hq_selftest_wait(0, 0x100, 1000, 0) == hq.HQ_ERR_UNSUPPORTED
    assert L.hq_selftest_wait(0, 0, 0, 0) == L.hq_selftest_wait(0, 0, 5_000_000_000, 0) == hq.HQ_ERR_SHAPE
