"""Row counts past what the kernels' 32-bit offsets reach are refused before any HIP call."""
import ctypes

import pytest

from moe_grouped_gemm_scales_amd.dg import _Epilogue, lib

f = ctypes.c_void_p(0x100000)      # 16-byte aligned, never dereferenced
UNSUPPORTED = -2


@pytest.mark.parametrize("M", [1 << 30, (1 << 31) - 128])
def test_contiguous_bf16_rows(M):
    """m_indices has 4 bytes a row and is read as one buffer: 2^30 rows would be a buffer of size 0, whose rows all
    read as expert 0's."""
    e = ctypes.byref(_Epilogue(None, 0, 2, None, None))
    assert lib.dg_m_grouped_bf16_gemm_nt_contiguous(f, f, f, None, f, M, 16, 64, 2, None) == UNSUPPORTED
    assert lib.dg_m_grouped_bf16_gemm_nt_contiguous_epilogue(f, f, f, e, f, M, 16, 64, 2, None) == UNSUPPORTED
    assert lib.dg_m_grouped_bf16_gemm_nn_contiguous(f, f, f, None, f, M, 16, 64, 2, None) == UNSUPPORTED
    assert lib.dg_m_grouped_bf16_gemm_nn_contiguous_k_tail(f, f, f, None, f, M, 16, 65, 2, None) == UNSUPPORTED
