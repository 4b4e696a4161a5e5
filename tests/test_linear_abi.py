"""Argument checks, on the CPU, of the products with a fused epilogue, their backward pass and the BF16 NN and
TN products: refused before any HIP call."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import _Epilogue, lib

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


def _ep(bias=FAKE, bias_type=0, activation=2, residual=FAKE, Z=FAKE):
    return ctypes.byref(_Epilogue(bias, bias_type, activation, residual, Z))


BAD_EPILOGUES = [(dict(bias_type=2), INVALID), (dict(activation=5), INVALID), (dict(activation=-1), INVALID),
                 (dict(bias=FAKE + 4), ALIGNMENT), (dict(residual=FAKE + 8), ALIGNMENT), (dict(Z=FAKE + 2), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", BAD_EPILOGUES)
def test_bad_epilogue(kw, status):
    e = _ep(**kw)
    f = P(FAKE)
    assert lib.dg_bf16_gemm_nt_epilogue(f, f, e, f, 64, 64, 64, None) == status
    assert lib.dg_fp8_gemm_nt_epilogue(f, f, f, f, e, f, 64, 64, 128, None) == status
    assert lib.dg_fp8_gemm_nt_ue8m0_epilogue(f, f, f, f, e, f, 64, 64, 128, None) == status
    for n in ("contiguous", "masked"):
        assert getattr(lib, f"dg_m_grouped_bf16_gemm_nt_{n}_epilogue")(f, f, f, e, f, 128, 64, 64, 2, None) == status
        assert getattr(lib, f"dg_m_grouped_fp8_gemm_nt_{n}_epilogue")(f, f, f, f, f, e, f, 128, 64, 128, 2, None) == status
        assert getattr(lib, f"dg_m_grouped_fp8_gemm_nt_{n}_ue8m0_epilogue")(f, f, f, f, f, e, f, 128, 64, 128, 2, None) == status
    assert lib.dg_last_error().decode()


def test_epilogue_forms_keep_the_checks_of_the_plain_ones():
    f, e = P(FAKE), _ep()
    assert lib.dg_bf16_gemm_nt_epilogue(f, f, None, f, 64, 64, 64, None) == INVALID          # no epilogue struct
    assert lib.dg_bf16_gemm_nt_epilogue(None, f, e, f, 64, 64, 64, None) == INVALID
    assert lib.dg_bf16_gemm_nt_epilogue(f, f, e, f, 64, 64, 96, None) == UNSUPPORTED         # K % 64
    assert lib.dg_bf16_gemm_nt_epilogue(f, P(FAKE + 4), e, f, 64, 64, 64, None) == ALIGNMENT
    assert lib.dg_bf16_gemm_nt_epilogue(f, f, e, f, 0, 64, 64, None) == 0                    # M = 0
    assert lib.dg_fp8_gemm_nt_epilogue(f, f, f, f, e, f, 64, 64, 192, None) == UNSUPPORTED   # K % 128
    assert lib.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(f, f, f, e, f, 100, 64, 64, 2, None) == ALIGNMENT
    assert lib.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(f, f, None, e, f, 128, 64, 64, 2, None) == INVALID
    assert lib.dg_m_grouped_bf16_gemm_nt_masked_epilogue(f, f, f, e, f, 128, 64, 64, 0, None) == INVALID
    assert lib.dg_m_grouped_fp8_gemm_nt_masked_epilogue(f, f, f, f, P(FAKE + 2), e, f, 128, 64, 128, 2, None) == ALIGNMENT


@pytest.mark.parametrize("kw,status", [
    (dict(dD=0), INVALID), (dict(Z=0), INVALID), (dict(act=7), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(dD=FAKE + 8), ALIGNMENT), (dict(Z=FAKE + 2), ALIGNMENT), (dict(dZ=FAKE + 4), ALIGNMENT),
    (dict(db=FAKE + 2), ALIGNMENT), (dict(N=2 ** 31 - 1), UNSUPPORTED)])
def test_epilogue_backward_refusals(kw, status):
    a = dict(dD=FAKE, Z=FAKE, act=3, dZ=FAKE, db=FAKE, M=128, N=64) | kw
    assert lib.dg_epilogue_backward(P(a["dD"]), P(a["Z"]), a["act"], P(a["dZ"]), P(a["db"]), a["M"], a["N"], None) == status
    assert lib.dg_m_grouped_epilogue_backward_contiguous(P(a["dD"]), P(a["Z"]), a["act"], P(FAKE), P(a["dZ"]), P(a["db"]),
                                                         a["M"], a["N"], 2, None) == status


def test_grouped_epilogue_backward_refusals():
    f = P(FAKE)
    g = lib.dg_m_grouped_epilogue_backward_contiguous
    assert g(f, f, 1, None, f, f, 128, 64, 2, None) == INVALID                 # m_indices
    assert g(f, f, 1, f, f, f, 100, 64, 2, None) == ALIGNMENT                  # M % 128
    assert g(f, f, 1, f, f, f, 128, 64, 0, None) == INVALID
    assert g(f, f, 1, P(FAKE + 1), f, f, 128, 64, 2, None) == ALIGNMENT
    assert g(f, f, 1, f, f, f, 128, 64, 70000, None) == UNSUPPORTED
    assert lib.dg_epilogue_backward(None, None, 0, None, None, 0, 64, None) == 0   # nothing to do


def test_backward_product_refusals():
    f = P(FAKE)
    assert lib.dg_bf16_gemm_nn(f, None, None, f, 64, 64, 64, None) == INVALID
    assert lib.dg_bf16_gemm_nn(f, f, None, f, 64, 64, 72, None) == UNSUPPORTED           # K % 64
    assert lib.dg_bf16_gemm_nn(f, f, P(FAKE + 8), f, 64, 64, 64, None) == ALIGNMENT
    assert lib.dg_m_grouped_bf16_gemm_nn_contiguous(f, f, f, None, f, 100, 64, 64, 2, None) == ALIGNMENT
    assert lib.dg_m_grouped_bf16_gemm_nn_contiguous(f, f, None, None, f, 128, 64, 64, 2, None) == INVALID
    assert lib.dg_bf16_gemm_tn(None, f, None, f, 64, 64, 64, None) == INVALID
    assert lib.dg_bf16_gemm_tn(f, f, None, None, 64, 64, 64, None) == INVALID
    assert lib.dg_bf16_gemm_tn(f, f, None, f, 64, 64, -1, None) == INVALID
    assert lib.dg_bf16_gemm_tn(f, P(FAKE + 4), None, f, 64, 64, 64, None) == ALIGNMENT
    assert lib.dg_bf16_gemm_tn(f, f, None, f, 64, 64, 2 ** 31 - 1, None) == UNSUPPORTED
    assert lib.dg_bf16_gemm_tn(f, f, None, f, 0, 64, 64, None) == 0                      # M = 0
    k = lib.dg_k_grouped_bf16_gemm_tn_contiguous
    assert k(f, f, None, None, f, 64, 64, 128, 2, None) == INVALID                       # ks
    assert k(f, f, f, None, f, 64, 64, 128, 0, None) == INVALID
    assert k(f, f, P(FAKE + 2), None, f, 64, 64, 128, 2, None) == ALIGNMENT
    assert k(f, f, f, None, f, 64, 64, 100, 2, None) == UNSUPPORTED                      # K % 128


def test_binding_refuses_wrong_tensors():
    a, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    d = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dg.dg_bf16_gemm_nt_epilogue(a.float(), w, d)
    with pytest.raises(ValueError):
        dg.dg_bf16_gemm_nt_epilogue(a, w, d)                       # host tensors
    with pytest.raises(ValueError):
        dg.dg_epilogue_backward(d, None, "swish", d, None)         # no such activation
    with pytest.raises(ValueError):
        dg.dg_epilogue_backward(d[0], None, "none", d, None)       # dD must be [M, N]


def test_more_rows_than_one_launch_holds():
    """128 rows a workgroup of 256 work items, of which a launch has fewer than 2^32."""
    f = P(FAKE)
    assert lib.dg_epilogue_backward(f, f, 1, f, f, (1 << 31) - 1, 8, None) == UNSUPPORTED
