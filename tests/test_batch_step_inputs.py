"""BatchStep refuses tensors that its calls, which take addresses, would read
past the end of or misread: wrong shapes, types and strides (host checks)."""
import pytest

torch = pytest.importorskip("torch")

from quantized_weight_matvec_hq_gb300 import batch_step  # noqa: E402
from quantized_weight_matvec_hq_gb300 import synthetic  # noqa: E402

SIZE = dict(n_experts=8, n_active=2, hidden=256, vocab=512, n_adapters=3)


def step_of(dtype="bf16"):
    """A step's sizes without its weights and buffers."""
    s = batch_step.BatchStep.__new__(batch_step.BatchStep)
    s.k, s.hidden, s.vocab, s.n_adapters, s.most = 2, 256, 512, 3, 32
    s.x_dtype, s.device = batch_step.TORCH_DTYPES[dtype], torch.device("cpu")
    return s


def inputs(dtype="bf16"):
    a = batch_step.random_inputs(synthetic.rng(5), [3, 0, 2], dtype=dtype, device="cpu", **SIZE)
    return dict(a, q=torch.zeros((5, 512)))


def test_inputs_as_documented_are_taken():
    for dtype in ("f32", "f16", "bf16"):
        step_of(dtype)._check_inputs(**inputs(dtype))
    step_of()._check_inputs(**dict(inputs(), temperature=None, q=None))
    bare = step_of()
    bare.n_adapters = 0
    bare._check_inputs(**dict(inputs(), adapter_ids=None))


@pytest.mark.parametrize("name", sorted(inputs()))
def test_wrong_inputs_are_refused(name):
    s, good = step_of(), inputs()
    t = good[name]
    wide = torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype)
    bad = [t[..., :-1].contiguous(), wide[..., ::2], t.to(torch.float64), t.to("meta")]
    if t.dtype == torch.bfloat16:
        bad.append(t.to(torch.float16))
    for b in bad:
        with pytest.raises(ValueError):
            s(**dict(good, **{name: b}))


def test_wrong_weights_and_adapters_are_refused():
    sizes = dict(n_experts=8, n_active=2, hidden=256, ffn=256, vocab=512, most_tokens=8)
    W = [torch.zeros(n // 32 * 34, dtype=torch.uint8) for n in (8 * 512 * 256, 8 * 256 * 256, 512 * 256)]
    adapters = (torch.zeros((3, 4, 256), dtype=torch.bfloat16), torch.zeros((3, 512, 4), dtype=torch.bfloat16), torch.zeros(3))
    for i in range(3):
        with pytest.raises(ValueError):
            batch_step.BatchStep(*[w[:-1] if j == i else w for j, w in enumerate(W)], adapters, **sizes)
        for wrong in (adapters[i].double(), adapters[i][:-1] if i else adapters[i][..., :-1]):
            with pytest.raises(ValueError):
                batch_step.BatchStep(*W, tuple(wrong if j == i else a for j, a in enumerate(adapters)), **sizes)
