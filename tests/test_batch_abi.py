"""The batched step's entry points without a GPU: argument checks happen on the
host before any launch, empty calls return at once, and the workspace sizes are
host arithmetic."""
import numpy as np
import pytest

from quantized_weight_matvec_hq_gb300 import build as hq_build

FAKE = 1 << 40                                  # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def hq():
    hq_build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    return hq


def moe(hq, W=FAKE, w_exp=FAKE, ids=FAKE, x=FAKE, per_slot=0, rw=FAKE, y=FAKE, E=8, k=2, rows=64, cols=256, T=5, dt=2,
        epi=0, ws=FAKE, ws_bytes=1 << 40):
    return hq.lib().hq_moe_matmul_q8_0(W, w_exp, ids, x, per_slot, rw, y, E, k, rows, cols, T, dt, epi, ws, ws_bytes, 0)


def lora(hq, W=FAKE, w_exp=FAKE, x=FAKE, ids=FAKE, A=FAKE, B=FAKE, s=FAKE, n=3, rank=16, y=FAKE, rows=64, cols=256, T=5,
         dt=2, ws=FAKE, ws_bytes=1 << 40, fn="hq_matmul_q8_0_adapters"):
    return getattr(hq.lib(), fn)(W, w_exp, x, ids, A, B, s, n, rank, y, rows, cols, T, dt, ws, ws_bytes, 0)


def test_moe_matmul_refusals(hq):
    for name in ("W", "w_exp", "ids", "x", "y"):
        assert moe(hq, **{name: 0}) == hq.HQ_ERR_NULL, name
    assert moe(hq, rw=0, epi=hq.HQ_MOE_EPI_COMBINE) == hq.HQ_ERR_NULL
    for bad in (dict(E=0), dict(E=65536), dict(k=0), dict(k=9), dict(rows=0), dict(rows=1 << 29), dict(cols=128),
                dict(cols=288), dict(T=-1), dict(T=(1 << 26) + 1), dict(per_slot=2),
                dict(rows=7, epi=hq.HQ_MOE_EPI_SWIGLU)):
        assert moe(hq, **bad) == hq.HQ_ERR_SHAPE, bad
    assert moe(hq, dt=3) == moe(hq, dt=-1) == hq.HQ_ERR_UNSUPPORTED
    assert moe(hq, epi=3) == moe(hq, epi=-1) == hq.HQ_ERR_UNSUPPORTED
    for bad in (dict(W=FAKE + 8), dict(x=FAKE + 8), dict(y=FAKE + 1), dict(y=FAKE + 2, dt=0), dict(ids=FAKE + 2),
                dict(w_exp=FAKE + 2), dict(rw=FAKE + 2, epi=hq.HQ_MOE_EPI_COMBINE)):
        assert moe(hq, **bad) == hq.HQ_ERR_ALIGN, bad
    assert moe(hq, T=0, W=0, x=0, y=0, ids=0, ws=0, ws_bytes=0) == hq.HQ_OK


def test_adapter_refusals(hq):
    for fn in ("hq_matmul_q8_0_adapters", "hq_matmul_q4_0_adapters"):
        for name in ("W", "w_exp", "x", "y", "ids", "A", "B", "s"):
            assert lora(hq, fn=fn, **{name: 0}) == hq.HQ_ERR_NULL, name
        for bad in (dict(n=-1), dict(rank=0), dict(rank=65), dict(rank=-1), dict(rows=0), dict(cols=0), dict(cols=320),
                    dict(T=-1), dict(T=(1 << 27) + 1)):
            assert lora(hq, fn=fn, **bad) == hq.HQ_ERR_SHAPE, bad
        assert lora(hq, fn=fn, dt=7) == hq.HQ_ERR_UNSUPPORTED
        for bad in (dict(W=FAKE + 2), dict(x=FAKE + 2), dict(A=FAKE + 2), dict(B=FAKE + 1), dict(s=FAKE + 2),
                    dict(ids=FAKE + 1), dict(y=FAKE + 1)):
            assert lora(hq, fn=fn, **bad) == hq.HQ_ERR_ALIGN, bad
        assert lora(hq, fn=fn, T=0, x=0, y=0, ids=0, ws=0, ws_bytes=0) == hq.HQ_OK


def test_softmax_and_verify_refusals(hq):
    L = hq.lib()
    assert L.hq_softmax_rows(0, 0, FAKE, 2, 100, 0, 0) == hq.HQ_ERR_NULL
    assert L.hq_softmax_rows(FAKE, 0, 0, 2, 100, 0, 0) == hq.HQ_ERR_NULL
    assert L.hq_softmax_rows(FAKE, 0, FAKE, -1, 100, 0, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_softmax_rows(FAKE, 0, FAKE, 2, 0, 0, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_softmax_rows(FAKE, 0, FAKE, 2, (1 << 22) + 1, 0, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_softmax_rows(FAKE, 0, FAKE, 2, 100, 5, 0) == hq.HQ_ERR_UNSUPPORTED
    assert L.hq_softmax_rows(FAKE + 2, 0, FAKE, 2, 100, 0, 0) == hq.HQ_ERR_ALIGN
    assert L.hq_softmax_rows(FAKE + 1, 0, FAKE, 2, 100, 2, 0) == hq.HQ_ERR_ALIGN
    assert L.hq_softmax_rows(FAKE, 0, FAKE + 2, 2, 100, 2, 0) == hq.HQ_ERR_ALIGN
    assert L.hq_softmax_rows(0, 0, 0, 0, 100, 0, 0) == hq.HQ_OK
    good = [FAKE] * 8 + [3, 4, 100, 0]
    names = ("p", "q", "drafts", "off", "u", "us", "acc", "tokens")
    for i, name in enumerate(names):
        if name != "q":
            assert L.hq_verify_drafts(*(good[:i] + [0] + good[i + 1:])) == hq.HQ_ERR_NULL, name
        assert L.hq_verify_drafts(*(good[:i] + [FAKE + 2] + good[i + 1:])) == hq.HQ_ERR_ALIGN, name
    for i, v in ((8, -1), (8, (1 << 24) + 1), (9, -1), (9, 1 << 30), (10, 0), (10, (1 << 22) + 1)):
        assert L.hq_verify_drafts(*(good[:i] + [v] + good[i + 1:])) == hq.HQ_ERR_SHAPE, (i, v)
    assert L.hq_verify_drafts(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 100, 0) == hq.HQ_OK


def test_weight_exponents_refusals(hq):
    L = hq.lib()
    assert L.hq_weight_exponents(8, 0, FAKE, 1, 4, 64, 0) == hq.HQ_ERR_NULL
    assert L.hq_weight_exponents(8, FAKE, 0, 1, 4, 64, 0) == hq.HQ_ERR_NULL
    assert L.hq_weight_exponents(75, FAKE, FAKE, 1, 4, 256, 0) == hq.HQ_ERR_UNSUPPORTED
    assert L.hq_weight_exponents(8, FAKE, FAKE, 0, 4, 64, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_weight_exponents(8, FAKE, FAKE, 1, 4, 48, 0) == hq.HQ_ERR_SHAPE
    assert L.hq_weight_exponents(4, FAKE + 8, FAKE, 1, 4, 64, 0) == hq.HQ_ERR_ALIGN


def test_workspace_is_host_arithmetic(hq):
    n = hq.hq_moe_matmul_workspace(8, 2, 64, 256, 0, 0, hq.HQ_DT_BF16, 0)
    assert n >= 0
    last = 0
    for T in (1, 7, 64, 1000, 100000):
        n = hq.hq_moe_matmul_workspace(128, 8, 1536, 2048, T, 0, hq.HQ_DT_BF16, hq.HQ_MOE_EPI_COMBINE)
        assert n >= last
        last = n
        assert hq.hq_matmul_adapters_workspace(64, 4096, 4096, T, hq.HQ_DT_F32) >= 0
    with pytest.raises(hq.HQError):
        hq.hq_moe_matmul_workspace(8, 9, 64, 256, 5, 0, 0, 0)
    with pytest.raises(hq.HQError):
        hq.hq_matmul_adapters_workspace(65, 64, 256, 5, 0)
    need = hq.hq_moe_matmul_workspace(8, 2, 64, 256, 5, 0, hq.HQ_DT_BF16, 0)
    if need:
        assert moe(hq, ws_bytes=need - 1) == hq.HQ_ERR_SHAPE
        assert moe(hq, ws=0, ws_bytes=need) == hq.HQ_ERR_NULL
        assert moe(hq, ws=FAKE + 16, ws_bytes=need) == hq.HQ_ERR_ALIGN


def test_positions_of_a_step():
    pytest.importorskip("torch")
    from quantized_weight_matvec_hq_gb300 import batch_step
    request, number = batch_step.positions(np.array([0, 2, 2, 5], np.int32))
    assert request.tolist() == [0, 0, 0, 1, 2, 2, 2, 2]
    assert number.tolist() == [0, 1, 2, 0, 0, 1, 2, 3]
