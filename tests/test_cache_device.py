"""The cache's and the step's device, without a GPU: calls run on the current device, so what lies on another is refused
before any call of the library."""
import pytest

torch = pytest.importorskip("torch")

from quantized_weight_matvec_hq_gb300 import build as hq_build  # noqa: E402


@pytest.fixture(scope="module")
def batch_step():
    hq_build.build()
    from quantized_weight_matvec_hq_gb300 import batch_step
    return batch_step


def test_the_current_device_alone(batch_step, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    batch_step._expect_current(torch.device("cuda", 1))
    for other in (torch.device("cuda", 0), torch.device("cuda", 2), torch.device("cpu"), torch.device("meta")):
        with pytest.raises(ValueError, match="current"):
            batch_step._expect_current(other)


def test_calls_on_another_device_are_refused(batch_step, monkeypatch):
    """Tensors as documented, on a device that is not the current one: nothing of the library is called."""
    for name in ("hq_cache_write", "hq_cache_read", "hq_cache_attention"):
        monkeypatch.setattr(batch_step.hq, name, lambda *a, **k: pytest.fail("called"))
    c = batch_step.KeyValueCache("q8_0", 6, 32, 2, 64, device="cpu")
    batch = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2), dtype=torch.int32)
    rows, q = torch.zeros((5, 2, 64)), torch.zeros((5, 4, 64))
    for call in (lambda: c.write(rows, rows, batch), lambda: c.read(rows, rows.clone(), batch),
                 lambda: c.attend(q, torch.zeros_like(q), batch, torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="current"):
            call()


def test_steps_on_another_device_are_refused(batch_step):
    from quantized_weight_matvec_hq_gb300 import synthetic
    size = dict(n_experts=8, n_active=2, hidden=256, vocab=512, n_adapters=3)
    s = batch_step.BatchStep.__new__(batch_step.BatchStep)
    s.k, s.hidden, s.vocab, s.n_adapters, s.most, s.attention = 2, 256, 512, 3, 32, None
    s.x_dtype, s.device = torch.float32, torch.device("cpu")
    with pytest.raises(ValueError, match="current"):
        s(**batch_step.random_inputs(synthetic.rng(5), [3, 0, 2], dtype="f32", device="cpu", **size))


def test_weights_on_another_device_are_refused(batch_step):
    W = [torch.zeros(n // 32 * 34, dtype=torch.uint8) for n in (8 * 512 * 256, 8 * 256 * 256, 512 * 256)]
    with pytest.raises(ValueError, match="current"):
        batch_step.BatchStep(*W, None, n_experts=8, n_active=2, hidden=256, ffn=256, vocab=512, most_tokens=8)
