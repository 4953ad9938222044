"""The example layer (examples/moe_layer.py) runs every mixture-of-experts call together with the block-scaled
grouped GEMM, against plain FP32 torch.

out: each product's two operands are rounded to e4m3, at most 2^-4 of each value: on random signs a
relative 2-norm error near 2^-4 / sqrt(3) = 0.036 per operand at most (the rounding error is spread over
its interval), sqrt(4) of that over two products, and the BF16 roundings far below: 0.08.  The loss and the
router's gradient are FP32 sums of at most 1024 terms: 2^-24 * 1024 = 6e-5, times 16 for the gradient's dot
products of cancelling terms."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=1, experts=8, top_k=2), dict(tokens=333, hidden=272, inner=400, experts=10, top_k=3),
                                   dict(tokens=2500, hidden=1024, inner=512, experts=4, top_k=2),
                                   dict(tokens=130, hidden=256, inner=256, experts=40, top_k=8, padded=30)])
def test_layer_against_plain_torch(example, sizes):
    error, loss_error, grad_error = example.run(**sizes)
    assert error <= 0.08, error
    assert loss_error <= 6e-5, loss_error
    assert grad_error <= 16 * 6e-5, grad_error
