"""Which rows the contiguous form of the epilogue's backward pass writes: those of the experts, and zeros in rows
marked -1.  A row with any other index outside [0, G) is padding too and stays as it was, whether or not a bias
gradient is asked for."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("padding", [3, 1000, 65535, 2 ** 31 - 1, -2, -2 ** 31])
@pytest.mark.parametrize("N", [64, 515])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_padding_marked_by_any_index_is_untouched(padding, N, act):
    G, m = 3, []
    for g, c in enumerate([100, 0, 130]):
        m += [g] * c + [padding] * (-c % 128)
    m = torch.tensor(m + [padding] * 128 + [-1] * 128, dtype=torch.int32)
    real = (m >= 0) & (m < G)
    dd, z = _bf((len(m), N), 1), _bf((len(m), N), 2)
    dd[~real] = float("nan")
    z[~real] = float("nan")
    out = []
    for bias in (True, False):
        dz = torch.full((len(m), N), float("inf"), dtype=torch.bfloat16, device="cuda")
        db = torch.empty((G, N), device="cuda") if bias else None
        dg.dg_epilogue_backward(dd.cuda(), z.cuda() if act != "none" else None, act, dz, db, m.cuda(), num_experts=G)
        out.append(dz.cpu())
    dz = out[0]
    assert torch.equal(out[1].view(torch.int16), dz.view(torch.int16))
    assert torch.isinf(dz[~real & (m != -1)].float()).all() and (dz[m == -1] == 0).all()
    d, zz = dd[real].double().numpy(), z[real].double().numpy()
    want = d * ref.slope(zz, act)
    # the bound of tests/test_gpu_linear.py
    assert np.all(np.abs(dz[real].double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(d) * (1 + np.abs(zz)))


def test_number_of_experts_is_checked():
    d = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(128, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):          # the bias gradient of two experts, of which there are three
        dg.dg_epilogue_backward(d, None, "none", d, torch.zeros((2, 64), device="cuda"), m, num_experts=3)
    for n in (0, -1, 70000):
        with pytest.raises(dg.DGError):
            dg.dg_epilogue_backward(d, None, "none", d, None, m, num_experts=n)
