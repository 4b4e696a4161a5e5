"""The example's block, two in a row: norm, router, experts with 8-bit kept pre-activations, forward and backward, against
32-bit autograd with the same choice of experts."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(300, 512, 384, 6, 2), (77, 256, 192, 5, 3), (1, 128, 128, 4, 1)])
def test_block_and_gradients(tokens, hidden, inner, experts, topk, activation):
    """BF16 keeps every step within 2^-8 or so of the 32-bit one.  A kept pre-activation is within 2^-4 of its own, which
    the activation and its slope pass on scaled by z act'(z) / act(z) and z act''(z) / act'(z), of size one around the
    values of these layers, element by element and without a common sign: in the 2-norm the gradients stay within 2^-4."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples.moe_layer import check_block
    for name, d in check_block(tokens, hidden, inner, experts, topk, activation).items():
        # a single choice has the constant weight 1: the router's gradient is zero, and its distance from rounding has no meaning
        if name.endswith(".router") and topk == 1:
            continue
        assert d < (2 ** -6 if name.endswith(".y") else 2 ** -4), (name, d)
