"""GPU tests of a layer's norm, routing and experts: calls that the header allows and that lie off the usual ones."""
import math

import pytest

import layer_plain as lp
from test_gpu_layer import Block, check_route, generator, near, qm  # noqa: F401 (a fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# ---- experts

@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("tokens", [3, 40, 170])  # few rows an expert, up to 24, more
def test_experts_whose_gate_is_up(qm, tokens, kind, dtype):  # noqa: F811
    """One tensor as gate and as up: act(W x) * (W x), not act(W x)."""
    b = Block(qm, 4, 512, 320, kind=kind, seed=kind + 30)
    b.gate = b.up
    b.handle = qm.Experts(b.up, b.up, b.down, activation=kind)
    b.check(*b.rows(tokens, 2, dtype))
