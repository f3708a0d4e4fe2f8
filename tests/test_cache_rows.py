"""The rows that KeyValueCache takes, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from quantized_weight_matvec_hq_gb300 import build as hq_build  # noqa: E402


def test_the_stride_of_one_token_does_not_matter():
    """A row of any wider matrix: where there is no next token, the distance to it is not the library's to refuse."""
    hq_build.build()
    from quantized_weight_matvec_hq_gb300 import batch_step
    c = batch_step.KeyValueCache("q4_0", 2, 16, 2, 64, device="cpu")
    for width in (128, 131, 4096):
        row = torch.zeros((3, width)).as_strided((1, 2, 64), (width, 64, 1))
        assert row.stride(0) == width and c._rows("k", row, 2)[1] == 128
    assert c._rows("k", torch.zeros((3, 131))[:, :128].unflatten(1, (2, 64)), 2)[1] == 131
