"""Argument checks of the norm's entry points on the CPU (refused before any HIP call), and its gradient's formula
against differences."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import _Norm, lib
from tests import layer_ref as ref

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


def _norm(**kw):
    a = dict(x=FAKE, residual=FAKE, weight=FAKE, weight_type=1, eps=1e-6, S=FAKE, Y=2 * FAKE, Q=3 * FAKE, sf=FAKE, ue8m0=0,
             T=4, H=256) | kw
    n = _Norm(*(a[k] for k in ("residual", "weight", "weight_type", "eps", "S", "Y", "Q", "sf", "ue8m0")))
    return lib.dg_rms_norm(P(a["x"]), ctypes.byref(n), a["T"], a["H"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(sf=None), INVALID), (dict(S=None, Y=None, Q=None), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(weight_type=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(S=FAKE, Y=FAKE), INVALID), (dict(H=200), UNSUPPORTED), (dict(H=32769, Q=None), UNSUPPORTED),
    (dict(T=1 << 30, H=128), UNSUPPORTED), (dict(x=FAKE + 8), ALIGNMENT), (dict(residual=FAKE + 2), ALIGNMENT),
    (dict(weight=FAKE + 4), ALIGNMENT), (dict(S=FAKE + 2), ALIGNMENT), (dict(Y=FAKE + 4), ALIGNMENT),
    (dict(Q=FAKE + 8), ALIGNMENT), (dict(sf=FAKE + 2), ALIGNMENT)])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status
    assert lib.dg_last_error().decode()


def test_norm_null_struct():
    assert lib.dg_rms_norm(P(FAKE), None, 4, 256, None) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(s=None), INVALID), (dict(dx=None, dw=None), INVALID), (dict(T=-1), INVALID),
    (dict(H=0), INVALID), (dict(weight_type=7), INVALID), (dict(eps=-1.0), INVALID), (dict(H=32769), UNSUPPORTED),
    (dict(dy=FAKE + 2), ALIGNMENT), (dict(s=FAKE + 8), ALIGNMENT), (dict(w=FAKE + 2), ALIGNMENT),
    (dict(ds=FAKE + 2), ALIGNMENT), (dict(dx=FAKE + 2), ALIGNMENT), (dict(dw=FAKE + 2), ALIGNMENT)])
def test_norm_backward_refusals(kw, status):
    a = dict(dy=FAKE, s=FAKE, w=FAKE, weight_type=1, eps=1e-6, ds=FAKE, dx=FAKE, dw=FAKE, T=4, H=256) | kw
    assert lib.dg_rms_norm_backward(P(a["dy"]), P(a["s"]), P(a["w"]), a["weight_type"], a["eps"], P(a["ds"]), P(a["dx"]),
                                    P(a["dw"]), a["T"], a["H"], None) == status
    assert lib.dg_last_error().decode()


def test_norm_of_no_rows_is_no_call():
    assert _norm(T=0) == 0 and _norm(T=0, x=None, S=None, Y=None, Q=None, residual=None) == 0
    assert lib.dg_rms_norm_backward(None, None, None, 0, 0.0, None, None, None, 0, 256, None) == 0


def test_norm_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dg.dg_rms_norm(x, None, 1e-6, Y=x)                                     # host tensors
    with pytest.raises(TypeError):
        dg.dg_rms_norm(x.float(), None, 1e-6, Y=x)
    with pytest.raises(ValueError):
        dg.dg_rms_norm(x.reshape(2, 2, 256), None, 1e-6, Y=x)                  # rows must be [T, H]
    with pytest.raises(ValueError):
        dg.dg_rms_norm_backward(x, x, None, 1e-6, x, None)


@pytest.mark.parametrize("weight,past", [(True, True), (False, False)])
def test_norm_gradient_against_differences(weight, past):
    """The 64-bit gradient's formula is the derivative of the 64-bit norm."""
    g = torch.Generator().manual_seed(1)
    T, H, eps, step = 3, 11, 1e-3, 1e-6
    s, dy, w, ds = (torch.randn(n, generator=g, dtype=torch.float64) for n in ((T, H), (T, H), (H,), (T, H)))
    w, ds = w if weight else None, ds if past else None

    def loss(s, w):
        return float((ref.rms_norm(s, None, w, eps)[1] * dy).sum() + (0 if ds is None else (s * ds).sum()))

    dx, dw, _, _ = ref.rms_norm_backward(dy, s, w, eps, ds)
    for t in range(T):
        for h in range(H):
            e = torch.zeros_like(s)
            e[t, h] = step
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * step) - float(dx[t, h])) < 1e-7
    if weight:
        for h in range(H):
            e = torch.zeros_like(w)
            e[h] = step
            assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * step) - float(dw[h])) < 1e-7
