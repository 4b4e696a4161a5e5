"""Activations and slopes far below zero, where the results are small: held to a relative bound.

One BF16 rounding (eight significant bits) is at most 2^-8 of the result.  In FP32 an exponent of up to 126 ln 2 is the product of at most four rounded
factors, 126 ln 2 * 4 * 2^-24 = 2.1e-5 of the result; with the few 2^-23 of exp2, the reciprocal and Phi's polynomial
that is under 2^-15.  Results under 2^-118 are left out: their factors pass FP32's smallest normal value."""
import numpy as np
import pytest
import torch
from scipy.special import erfc, expit

import moe_grouped_gemm_scales_amd as dg
from tests import check

pytestmark = pytest.mark.gpu
FP32 = 2.0 ** -15
SMALL = 2.0 ** -118
C = np.sqrt(2 / np.pi)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _z(lowest):
    return torch.linspace(lowest, -1, 4000).to(torch.bfloat16).unique()


def _act(z, name):
    if name == "silu":
        return z * expit(z)
    if name == "gelu":
        return 0.5 * z * erfc(-z / np.sqrt(2))
    return z * expit(2 * C * (z + 0.044715 * z ** 3))


def _slope(z, name):
    """(slope, sum of the magnitudes of its two terms)"""
    if name == "silu":
        s, t = expit(z), z * expit(z) * expit(-z)
    elif name == "gelu":
        s, t = 0.5 * erfc(-z / np.sqrt(2)), z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    else:
        s = expit(2 * C * (z + 0.044715 * z ** 3))
        t = z * s * expit(-2 * C * (z + 0.044715 * z ** 3)) * 2 * C * (1 + 3 * 0.044715 * z * z)
    return s + t, np.abs(s) + np.abs(t)


CASES = [("silu", -80.0), ("gelu", -12.5), ("gelu_tanh", -9.5)]


@pytest.mark.parametrize("act,lowest", CASES)
@pytest.mark.parametrize("N", [32, 33, 35])
def test_forward(act, lowest, N):
    z = _z(lowest)
    A, B = torch.zeros((len(z), 64), dtype=torch.bfloat16), torch.zeros((N, 64), dtype=torch.bfloat16)
    A[:, 0], B[:, 0] = z, 1
    D = torch.empty((len(z), N), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_gemm_nt_epilogue(A.cuda(), B.cuda(), D, activation=act)
    want = _act(z.double().numpy(), act)
    got = check.bf16_to_f64(D.cpu())
    assert (got == got[:, :1]).all()
    keep = np.abs(want) > SMALL
    assert keep.sum() > 300
    rel = np.abs(got[keep, 0] / want[keep] - 1)
    assert rel.max() <= 2.0 ** -8 + FP32, (z[torch.from_numpy(keep)][rel.argmax()], rel.max())


@pytest.mark.parametrize("act,lowest", CASES)
def test_slope(act, lowest):
    z = _z(lowest)[None]
    db = torch.empty(z.shape[1], device="cuda")
    dg.dg_epilogue_backward(torch.ones_like(z).cuda(), z.cuda(), act, None, db)
    want, size = _slope(z[0].double().numpy(), act)
    keep = np.abs(want) > SMALL
    err = np.abs(db.cpu().double().numpy() - want)[keep] / size[keep]
    assert err.max() <= FP32, (z[0][torch.from_numpy(keep)][err.argmax()], err.max())
