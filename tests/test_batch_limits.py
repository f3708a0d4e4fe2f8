"""Sizes at the limits of the batched step's calls, refused on the host with
the status that the header names, by a call and by its workspace function."""
import pytest

from quantized_weight_matvec_hq_gb300 import build as hq_build

FAKE = 1 << 40                                  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hq():
    hq_build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    return hq


def test_workspaces_refuse_what_the_calls_refuse(hq):
    L = hq.lib()
    rows, T = 1 << 20, 1 << 27                  # 2^13 row tiles of 2^23 token tiles
    assert L.hq_matmul_adapters_workspace(16, rows, 256, T, 2) == hq.HQ_ERR_SHAPE
    for fn in (L.hq_matmul_q8_0_adapters, L.hq_matmul_q4_0_adapters):
        assert fn(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 3, 16, FAKE, rows, 256, T, 2, FAKE, 1 << 62, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_moe_matmul_workspace(8, 2, rows, 256, T // 2, 0, 2, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_moe_matmul_q8_0(FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, 8, 2, rows, 256, T // 2, 2, 0, FAKE, 1 << 62, 0) == hq.HQ_ERR_SHAPE
    # the largest that fit
    assert L.hq_matmul_adapters_workspace(16, 255 * 128, 256, T, 2) > 0
    assert L.hq_moe_matmul_workspace(8, 2, 255 * 128, 256, T // 2, 0, 2, 0) > 0


def test_softmax_refuses_more_rows_than_a_grid_has(hq):
    L = hq.lib()
    for rows in (1 << 28, (1 << 28) + 1):
        assert L.hq_softmax_rows(FAKE, 0, FAKE, rows, 100, 0, 0) == hq.HQ_ERR_SHAPE
