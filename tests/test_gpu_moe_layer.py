"""The example layer end to end: forward and backward in BF16, and the FP8 decode path, against the same
layer in 32-bit torch operations with autograd.

Bounds, as the 2-norm of the difference over that of the result.  BF16: a forward value passes at most four
BF16 roundings (h, out, y, and Z for the gradients), a gradient at most six; each is at most 2^-9 rms of its
value, so 6 * 2^-9 = 1.2e-2 holds all of them even if they added up.  FP8: both operands of both products
carry E4M3's relative error, at most 2^-4 and 2^-4 / sqrt(3) rms for the value nearest a power of two: four
such operands give at most 4 * 2^-4 / sqrt(3) = 0.145."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


@pytest.mark.parametrize("kw", [dict(), dict(tokens=1, experts=3, topk=2), dict(tokens=77, experts=9, topk=4, activation="silu"),
                                dict(tokens=513, hidden=256, inner=640, experts=2, topk=1, activation="gelu_tanh")])
def test_layer_against_torch(kw):
    from examples.moe_layer import check
    for name, far in check(**kw).items():
        assert far <= (0.145 if name == "y_fp8" else 1.2e-2), (name, far)
