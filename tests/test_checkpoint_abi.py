"""Argument checks of the 8-bit checkpoint entry points on the CPU: refused before any HIP call."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import lib

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(M=-1), INVALID),
    (dict(N=0), INVALID), (dict(N=(1 << 31) - 1, M=1), UNSUPPORTED), (dict(M=1 << 30, N=256), UNSUPPORTED),
    (dict(x=FAKE + 8), ALIGNMENT), (dict(codes=FAKE + 4), ALIGNMENT), (dict(m=FAKE + 2), ALIGNMENT)])
def test_keep_and_restore_refusals(kw, status):
    a = dict(x=FAKE, codes=FAKE, scales=FAKE, m=FAKE, M=4, N=256) | kw
    assert lib.dg_checkpoint_fp8(P(a["x"]), P(a["m"]), P(a["codes"]), P(a["scales"]), a["M"], a["N"], None) == status
    assert lib.dg_last_error().decode()
    assert lib.dg_checkpoint_restore(P(a["codes"]), P(a["scales"]), P(a["m"]), P(a["x"]), a["M"], a["N"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dd=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(M=-128), INVALID),
    (dict(N=0), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(h=FAKE), INVALID),
    (dict(h=2 * FAKE), INVALID), (dict(N=65536 * 512), UNSUPPORTED), (dict(dd=FAKE + 8), ALIGNMENT),
    (dict(codes=FAKE + 8), ALIGNMENT), (dict(dz=FAKE + 2), ALIGNMENT), (dict(h=FAKE + 2), ALIGNMENT),
    (dict(db=FAKE + 2), ALIGNMENT)])
def test_backward_refusals(kw, status):
    a = dict(dd=FAKE, codes=FAKE, scales=FAKE, act=2, dz=2 * FAKE, h=3 * FAKE, db=FAKE, M=128, N=256) | kw
    args = (P(a["dd"]), P(a["codes"]), P(a["scales"]), a["act"])
    out = (P(a["dz"]), P(a["h"]), P(a["db"]), a["M"], a["N"])
    assert lib.dg_epilogue_backward_fp8(*args, *out, None) == status
    assert lib.dg_last_error().decode()
    assert lib.dg_m_grouped_epilogue_backward_fp8_contiguous(*args, P(FAKE), *out, 4, None) == status


def test_grouped_backward_refusals():
    f = P(FAKE)
    call = lib.dg_m_grouped_epilogue_backward_fp8_contiguous
    assert call(f, f, f, 2, None, f, None, None, 128, 256, 4, None) == INVALID
    assert call(f, f, f, 2, P(FAKE + 2), f, None, None, 128, 256, 4, None) == ALIGNMENT
    assert call(f, f, f, 2, f, f, None, None, 100, 256, 4, None) == ALIGNMENT
    assert call(f, f, f, 2, f, f, None, None, 128, 256, 0, None) == INVALID
    assert call(f, f, f, 2, f, f, None, None, 128, 256, 65536, None) == UNSUPPORTED


def test_checkpoint_of_no_rows_is_no_call():
    assert lib.dg_checkpoint_fp8(None, None, None, None, 0, 256, None) == 0
    assert lib.dg_checkpoint_restore(None, None, None, None, 0, 256, None) == 0
    assert lib.dg_epilogue_backward_fp8(None, None, None, 2, None, None, None, 0, 256, None) == 0


def test_checkpoint_binding_refuses_wrong_tensors():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    c, s = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError):
        dg.dg_checkpoint_fp8(x, c, s)                                # host tensors
    with pytest.raises(TypeError):
        dg.dg_checkpoint_restore(c, s, x.float())
    with pytest.raises(ValueError):
        dg.dg_epilogue_backward_fp8(x, c, s, "swish", x, None)
