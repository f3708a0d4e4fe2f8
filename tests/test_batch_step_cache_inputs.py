"""The step's cache without a GPU: tensors of other shapes, types, strides or devices than documented are refused before
any call of the library (its calls take addresses)."""
import pytest

torch = pytest.importorskip("torch")

from quantized_weight_matvec_hq_gb300 import build as hq_build  # noqa: E402


@pytest.fixture(scope="module")
def cache():
    hq_build.build()
    from quantized_weight_matvec_hq_gb300 import batch_step
    return batch_step.KeyValueCache("q4_0", 6, 32, 2, 64, device="cpu")


def batch(R=3, W=2):
    return torch.zeros(R + 1, dtype=torch.int32), torch.zeros(R, dtype=torch.int32), torch.zeros((R, W), dtype=torch.int32)


def test_the_pool_has_the_pages(cache):
    assert cache.pool.numel() == 6 * 2 * 2 * 32 * 2 * 18


def test_rows_are_refused(cache):
    good = torch.zeros((5, 2, 64))
    wide = torch.zeros((5, 9, 64))
    assert cache._rows("k", wide[:, 3:5], 2)[1] == 9 * 64
    assert cache._rows("k", good[:1], 2)[1] == 2 * 64 and cache._rows("k", good[:0], 2)[1] == 2 * 64
    for bad in (good[:, :1], good[..., :32], good.transpose(0, 1), good.to(torch.float64), good.flatten(1), good[..., ::2],
                torch.zeros((5, 4, 64))[:, ::2], good.to("meta")):
        with pytest.raises(ValueError):
            cache.write(bad, bad, batch())
        with pytest.raises(ValueError):
            cache.read(bad, bad, batch())
    with pytest.raises(ValueError):
        cache.write(good, good[:4], batch())
    with pytest.raises(ValueError):
        cache.write(good, good.half(), batch())


def test_batches_are_refused(cache):
    rows = torch.zeros((5, 2, 64))
    o, l, t = batch()
    for bad in ((o[:3], l, t), (o, l[:2], t), (o, l, t[:2]), (o.long(), l, t), (o, l.float(), t), (o, l, t.t()), (o, l, t[:, ::2]),
                (o, l.to("meta"), t)):
        with pytest.raises(ValueError):
            cache.write(rows, rows, bad)
        with pytest.raises(ValueError):
            cache.attend(torch.zeros((5, 4, 64)), torch.zeros((5, 4, 64)), bad, torch.zeros(1 << 20, dtype=torch.uint8))


def test_attention_tensors_are_refused(cache):
    q, ws = torch.zeros((5, 4, 64)), torch.zeros(1 << 20, dtype=torch.uint8)
    for a in (dict(out=torch.zeros((5, 2, 64))), dict(out=torch.zeros((4, 4, 64))), dict(out=q.half()), dict(ws=ws.int()),
              dict(ws=ws[::2])):
        with pytest.raises(ValueError):
            cache.attend(q, a.get("out", torch.zeros_like(q)), batch(), a.get("ws", ws))


def test_pages_are_refused(cache):
    import numpy as np
    from quantized_weight_matvec_hq_gb300 import batch_step
    g = np.random.default_rng(0)
    lengths, table = batch_step.random_cache(g, cache, [33, 0, 64], 2)
    used = [int(table[0, 0]), int(table[0, 1]), int(table[2, 0]), int(table[2, 1])]
    assert lengths.tolist() == [33, 0, 64] and len(set(used)) == 4
    for lengths in ([65], [64, 64, 64, 1]):
        with pytest.raises(ValueError):
            batch_step.random_cache(g, cache, lengths, 2)


def test_position_offsets():
    from quantized_weight_matvec_hq_gb300 import batch_step
    assert batch_step.position_offsets(torch.tensor([0, 2, 2, 5], dtype=torch.int32)).tolist() == [0, 3, 4, 8]
