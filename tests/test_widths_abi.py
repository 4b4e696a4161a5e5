"""Argument checks, on the CPU, of the NN products of any K, and what they select."""
import ctypes

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import lib

f = ctypes.c_void_p(0x100000)      # 16-byte aligned, never dereferenced
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


def test_refusals():
    off = ctypes.c_void_p(0x100008)
    nn = lib.dg_bf16_gemm_nn_k_tail
    assert nn(None, f, None, f, 64, 64, 72, None) == INVALID
    assert nn(f, None, None, f, 64, 64, 72, None) == INVALID
    assert nn(f, f, None, None, 64, 64, 72, None) == INVALID
    assert nn(f, f, None, f, 64, 0, 72, None) == INVALID
    assert nn(f, f, None, f, 64, 64, 0, None) == INVALID
    assert nn(f, f, off, f, 64, 64, 72, None) == ALIGNMENT
    assert nn(f, off, None, f, 64, 64, 72, None) == ALIGNMENT
    assert nn(f, f, None, f, 64, 64, 2 ** 31 - 1, None) == UNSUPPORTED
    assert nn(None, f, None, None, 0, 64, 72, None) == 0                     # no rows
    g = lib.dg_m_grouped_bf16_gemm_nn_contiguous_k_tail
    assert g(f, f, None, None, f, 128, 64, 72, 2, None) == INVALID           # m_indices
    assert g(f, f, f, None, f, 100, 64, 72, 2, None) == ALIGNMENT            # M % 128
    assert g(f, f, f, None, f, 128, 64, 72, 0, None) == INVALID
    assert g(None, f, None, None, None, 0, 64, 72, 2, None) == 0


def test_selection():
    """The kernel of the whole K blocks, with both operands K-contiguous."""
    for kind, M, G in ((0, 300, 1), (1, 1024, 4)):
        key = dg.describe_config(kind | dg.KIND_BF16 | dg.LAYOUT_NN, M, 520, 1000, G, num_cus=256)
        assert "_K2048_" in key and "_nn" not in key, key
        assert "_nn" in dg.describe_config(kind | dg.KIND_BF16 | dg.LAYOUT_NN, M, 520, 1024, G, num_cus=256)
