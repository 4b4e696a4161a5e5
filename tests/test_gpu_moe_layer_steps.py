"""Steps of the example's training layer that follow a bad one: its row buffers are kept from step to step, so a row
that is padding in this step may hold what an earlier step left there."""
import pytest
import torch

from examples.moe_layer import BF16, MoELayer, distance, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_step_after_one_that_overflowed(bad, activation):
    """Step 1: all tokens to experts 0 and 1, some of them not finite.  Step 2: finite tokens, other routes, so that
    rows in use before are padding now.  Its gradients are finite and those of a fresh layer."""
    T, hidden, inner, E = 260, 128, 192, 4
    layer = MoELayer(T, hidden, inner, E, 2, activation, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda: torch.randn((T, hidden), generator=g, device="cuda").to(BF16)
    weights = torch.full((T, 2), 0.5, device="cuda")
    x, dy = rnd(), rnd()
    x[::3] = bad
    layer.forward(x, torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda"), weights)
    layer.backward(dy)
    x, dy = rnd(), rnd()
    ids = torch.tensor([[t % 4, (t + 1) % 4] for t in range(T)], dtype=torch.int32, device="cuda")
    y = layer.forward(x, ids, weights)
    grads = layer.backward(dy)
    fresh = MoELayer(T, hidden, inner, E, 2, activation, seed=3)
    assert torch.equal(fresh.forward(x, ids, weights), y)
    for name, v in fresh.backward(dy).items():
        assert torch.isfinite(grads[name].float()).all(), name
        assert torch.equal(grads[name], v), name
    want, v = reference(layer, x, ids, weights)
    want.backward(dy.float())
    for n in v:                                # the bound of tests/test_gpu_moe_layer.py
        assert distance(grads[n], v[n].grad) <= 1.2e-2, n
