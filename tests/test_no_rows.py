"""Calls without rows.  torch's empty tensors have no address, so the arrays that have no elements may be NULL: the
products do nothing, a weight gradient over no rows is zero (or C).  The arrays that do have elements are checked as ever."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import _Epilogue, lib

P = ctypes.c_void_p
F = P(0x100000)          # 16-byte aligned, never dereferenced
INVALID = -1


def _ep():
    return ctypes.byref(_Epilogue(0x100000, 0, 2, None, None))


def _calls(B=F, groups=F):
    """Every form without rows: [(name, status)]; A, its scales, D and the rows' own indices NULL."""
    e, out = _ep(), []
    for n, sf in (("bf16", ()), ("fp8", (F,))):
        for tail, k in (("", 64 * (1 + len(sf))),):
            nul = tuple(None for _ in sf)
            g = lambda form, end: getattr(lib, f"dg_{'m_grouped_' if form != 'dense' else ''}{n}_gemm_nt{'' if form == 'dense' else '_' + form}{end}")
            out += [(f"{n} dense", g("dense", "")(None, *nul, B, *sf, None, None, 0, 64, k, None)),
                    (f"{n} dense epilogue", g("dense", "_epilogue")(None, *nul, B, *sf, e, None, 0, 64, k, None)),
                    (f"{n} contiguous", g("contiguous", "")(None, *nul, B, *sf, None, None, None, 0, 64, k, 2, None)),
                    (f"{n} contiguous epilogue", g("contiguous", "_epilogue")(None, *nul, B, *sf, None, e, None, 0, 64, k, 2, None)),
                    (f"{n} masked", g("masked", "")(None, *nul, B, *sf, groups, None, None, 0, 64, k, 2, None)),
                    (f"{n} masked epilogue", g("masked", "_epilogue")(None, *nul, B, *sf, groups, e, None, 0, 64, k, 2, None))]
    out += [("nn", lib.dg_bf16_gemm_nn(None, B, None, None, 0, 64, 64, None)),
            ("nn contiguous", lib.dg_m_grouped_bf16_gemm_nn_contiguous(None, B, None, None, None, 0, 64, 64, 2, None)),
            ("tn", lib.dg_bf16_gemm_tn(None, B, None, None, 0, 64, 64, None)),
            ("k-grouped tn", lib.dg_k_grouped_bf16_gemm_tn_contiguous(None, B, F, None, None, 0, 64, 128, 2, None))]
    return out


def test_no_rows_is_no_call():
    for name, status in _calls():
        assert status == 0, (name, lib.dg_last_error())


def test_arrays_with_elements_are_still_checked():
    for name, status in _calls(B=None):
        assert status == INVALID, name
    for name, status in _calls(groups=None):
        assert (status == INVALID) == ("masked" in name), name


@pytest.mark.gpu
@pytest.mark.parametrize("activation", ["none", "gelu"])
def test_layer_of_no_tokens(activation):
    """Forward, gradients and FP8 forward of the example layer for a step (or a rank) without tokens, then with some."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples.moe_layer import BF16, MoELayer, ServingLayer
    layer = MoELayer(0, 128, 256, 3, 2, activation)
    x, ids = torch.empty((0, 128), dtype=BF16, device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((0, 2), device="cuda")
    assert layer.rows.numel() == 0 and layer.forward(x, ids, w).shape == (0, 128)
    for name, g in layer.backward(x).items():
        assert not g.float().abs().sum(), name
    assert ServingLayer(layer, 16).forward(x, ids, w).shape == (0, 128)


@pytest.mark.gpu
def test_k_grouped_product_of_no_rows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    e = lambda n: torch.empty((0, n), dtype=torch.bfloat16, device="cuda")
    for M, N in ((40, 24), (264, 520), (33, 515)):
        D = torch.full((3, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        ks = torch.zeros(3, dtype=torch.int32, device="cuda")
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(e(M), e(N), ks, None, D)
        assert not D.float().abs().sum()
        C = torch.randn((3, M, N), device="cuda")
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(e(M), e(N), ks, C, D)
        assert torch.equal(D, C.to(torch.bfloat16))
