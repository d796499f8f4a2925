"""What the binding of a layer's experts refuses before it looks at the tensors."""
import pytest

import bit_block_quantized_qm_gb300 as qm

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("w_up", [None, [[1]], 3, b"1234"])
def test_experts_without_a_tensor(w_up):
    w = torch.zeros((2, 32, 18), dtype=torch.uint8)
    with pytest.raises(TypeError):
        qm.Experts(w, w_up, w)


@pytest.mark.parametrize("shape", [(), (64,), (32, 18), (1, 2, 32, 18)])
def test_experts_of_other_dimensions(shape):
    w = torch.zeros((2, 32, 18), dtype=torch.uint8)
    with pytest.raises(ValueError):
        qm.Experts(w, torch.zeros(shape, dtype=torch.uint8), w)
