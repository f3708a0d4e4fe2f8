"""The attention's workspace without a GPU: sizes are host arithmetic."""
import pytest

from quantized_weight_matvec_hq_gb300 import build as hq_build


@pytest.fixture(scope="module")
def hq():
    hq_build.build()
    import quantized_weight_matvec_hq_gb300 as hq
    hq.lib()
    return hq


def size(hq, R, T, dim=128, dtype="bf16", heads=32, kv=8):
    return hq.hq_cache_attention_workspace(4, 64, 1 << 12, R, T, heads, kv, dim, hq.DTYPE_CODES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_no_more_than_the_blocks_that_fit(hq, dim, dtype):
    """Two partial results of 128 rows (f32: 16) of every block on 152 multiprocessors, of which shared memory holds two, or one of
    heads of 256."""
    rows, blocks = (128, 1 if dim == 256 else 2) if dtype == "bf16" else (16, 4)
    need = 2 * 152 * blocks * rows * (dim + 2) * 4
    assert size(hq, 1, 4000, dim, dtype) <= need + 152 * blocks * 128
    if dtype == "bf16":
        assert size(hq, 1, 4000, dim, dtype) >= need


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,kv", [(32, 8), (8, 8), (9, 1), (16, 1), (64, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_larger_batch_s_serves_a_smaller_one(hq, dim, heads, kv, dtype):
    """Whatever kernel either takes: fewer tokens or requests never need more."""
    batches = [(R, T) for R in (1, 2, 3, 8, 64, 1000) for T in (1, 2, 3, 5, 8, 9, 16, 20, 64, 129, 4000)]
    need = {(R, T): size(hq, R, T, dim, dtype, heads, kv) for R, T in batches}
    for R, T in batches:
        assert 0 < need[R, T] < 41 * 2 ** 20
        for r, t in batches:
            assert r > R or t > T or need[r, t] <= need[R, T], ((r, t), (R, T))
