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


def test_binding_refuses_sizes_past_31_bits():
    """ctypes passes a size on modulo 2^32: 2^32 + 5 rows would be 5.  (meta tensors: no memory)"""
    import torch

    import moe_grouped_gemm_scales_amd as dg
    n = (1 << 32) + 128
    t = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")
    i = lambda *s: t(*s, dtype=torch.int32)
    calls = [lambda: dg.dg_moe_combine(t(8, 1), i(n, 2), None, None, t(n, 1)),
             lambda: dg.dg_moe_combine(t(n, 1), i(8, 2), None, None, t(8, 1)),
             lambda: dg.dg_moe_combine(t(1 << 16, 1 << 16, 1), i(8, 2), None, None, t(8, 1)),
             lambda: dg.dg_moe_dispatch_bf16(t(n, 1), i(n, 1), None, t(8, 1)),
             lambda: dg.dg_moe_dispatch_bf16(t(8, 1), i(8, 1), i(n), t(n, 1)),
             lambda: dg.dg_moe_dispatch_fp8(t(8, 128), i(8, 1), None, t(n, 128, dtype=torch.uint8), t(1, n, dtype=torch.float32)),
             lambda: dg.dg_moe_combine_backward(t(n, 1), None, i(n, 1), None, None, t(8, 1), None),
             lambda: dg.dg_epilogue_backward(t(n, 1), None, "none", t(n, 1), None),
             lambda: dg.dg_epilogue_backward(t(1, n), None, "none", t(1, n), None),
             lambda: dg.moe_sorted_rows(n, 1, 4)]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()
            raise AssertionError(k)
    with pytest.raises(ValueError, match=r"2\^31"):
        dg.dg_moe_sort_masked(i(n, 1), 4, 16, i(n, 1), i(4))
    with pytest.raises(ValueError, match=r"2\^31"):
        dg.dg_moe_sort_masked(i(8, 1), 4, n, i(8, 1), i(4))
