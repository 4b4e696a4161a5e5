"""Argument checks of the token sorting, dispatch and combine entry points on the CPU: refused before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import lib
from tests import moe_ref as ref

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


def test_sorted_rows_holds_every_choice():
    for T, k, G in [(0, 1, 1), (1, 1, 1), (1, 8, 32), (5, 3, 4), (1000, 2, 7), (33, 4, 1024)]:
        R = dg.moe_sorted_rows(T, k, G)
        assert R % 128 == 0 and R == ref.sorted_rows(T, k, G)
        for seed in range(3):
            rng = np.random.default_rng(seed)
            ids = rng.integers(0, G, (T, k)).astype(np.int32)
            _, _, ks = ref.sort_contiguous(ids, G, R + 128 * G)
            assert ks.sum() <= R
    with pytest.raises(ValueError):
        dg.moe_sorted_rows(-1, 2, 3)
    with pytest.raises(ValueError):
        dg.moe_sorted_rows(4, 0, 3)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=0), INVALID), (dict(pos=0), INVALID), (dict(m=0), INVALID), (dict(ks=0), INVALID), (dict(T=-1), INVALID),
    (dict(k=0), INVALID), (dict(G=0), INVALID), (dict(rows=-128), INVALID), (dict(G=1025), UNSUPPORTED),
    (dict(T=1 << 30, k=2), UNSUPPORTED), (dict(rows=100), ALIGNMENT), (dict(ids=FAKE + 2), ALIGNMENT),
    (dict(ks=FAKE + 1), ALIGNMENT)])
def test_sort_contiguous_refusals(kw, status):
    a = dict(ids=FAKE, pos=FAKE, m=FAKE, ks=FAKE, T=4, k=2, G=8, rows=1024) | kw
    assert lib.dg_moe_sort_contiguous(P(a["ids"]), P(a["pos"]), P(a["m"]), P(a["ks"]), a["T"], a["k"], a["G"], a["rows"],
                                      None) == status
    assert lib.dg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(ids=0), INVALID), (dict(mm=0), INVALID), (dict(m_max=0), INVALID), (dict(G=2000), UNSUPPORTED),
    (dict(m_max=1 << 30, G=4), UNSUPPORTED), (dict(mm=FAKE + 3), ALIGNMENT)])
def test_sort_masked_refusals(kw, status):
    a = dict(ids=FAKE, pos=FAKE, mm=FAKE, T=4, k=2, G=8, m_max=64) | kw
    assert lib.dg_moe_sort_masked(P(a["ids"]), P(a["pos"]), P(a["mm"]), a["T"], a["k"], a["G"], a["m_max"],
                                  None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), INVALID), (dict(pos=0), INVALID), (dict(out=0), INVALID), (dict(sf=0), INVALID), (dict(T=-1), INVALID),
    (dict(k=0), INVALID), (dict(H=0), INVALID), (dict(rows=-1), INVALID), (dict(H=200), UNSUPPORTED),
    (dict(group=100), INVALID), (dict(group=0), INVALID), (dict(x=FAKE + 8), ALIGNMENT), (dict(out=FAKE + 4), ALIGNMENT),
    (dict(sf=FAKE + 2), ALIGNMENT), (dict(m=FAKE + 2), ALIGNMENT), (dict(T=1 << 30, H=1 << 20), UNSUPPORTED)])
def test_dispatch_refusals(kw, status):
    a = dict(x=FAKE, pos=FAKE, m=None, out=FAKE, sf=FAKE, T=4, k=2, rows=256, group=256, H=256) | kw
    assert lib.dg_moe_dispatch_fp8(P(a["x"]), P(a["pos"]), P(a["m"]), P(a["out"]), P(a["sf"]), a["T"], a["k"], a["rows"],
                                   a["group"], a["H"], 0, None) == status
    if not {"sf", "group"} & set(kw) and kw.get("H") != 200:
        assert lib.dg_moe_dispatch_bf16(P(a["x"]), P(a["pos"]), P(a["m"]), P(a["out"]), a["T"], a["k"], a["rows"], a["H"],
                                        None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=0), INVALID), (dict(rows_in=0), INVALID), (dict(pos=0), INVALID), (dict(N=0), INVALID), (dict(k=-2), INVALID),
    (dict(y=FAKE + 8), ALIGNMENT), (dict(rows_in=FAKE + 2), ALIGNMENT), (dict(w=FAKE + 2), ALIGNMENT),
    (dict(res=FAKE + 8), ALIGNMENT), (dict(T=1 << 30, N=1 << 20), UNSUPPORTED)])
def test_combine_refusals(kw, status):
    a = dict(rows_in=FAKE, pos=FAKE, w=FAKE, res=None, y=FAKE, T=4, k=2, rows=256, N=64) | kw
    assert lib.dg_moe_combine(P(a["rows_in"]), P(a["pos"]), P(a["w"]), P(a["res"]), P(a["y"]), a["T"], a["k"], a["rows"],
                              a["N"], None) == status
    if not {"res", "T"} & set(kw) and "rows_in" not in kw:
        assert lib.dg_moe_combine_backward(P(a["y"]), P(FAKE), P(a["pos"]), P(a["w"]), None, P(FAKE), P(FAKE), a["T"],
                                           a["k"], a["rows"], a["N"], None) == status


def test_combine_backward_needs_rows_for_the_weights():
    assert lib.dg_moe_combine_backward(P(FAKE), None, P(FAKE), None, None, P(FAKE), P(FAKE), 4, 2, 256, 64, None) == INVALID


def test_nothing_to_do_is_no_call():
    """No tokens (and no rows to clear): DG_OK without a launch."""
    assert lib.dg_moe_dispatch_bf16(P(FAKE), P(FAKE), None, P(FAKE), 0, 2, 256, 64, None) == 0
    assert lib.dg_moe_dispatch_fp8(P(FAKE), P(FAKE), None, P(FAKE), P(FAKE), 0, 2, 256, 256, 128, 0, None) == 0
    assert lib.dg_moe_combine(P(FAKE), P(FAKE), None, None, P(FAKE), 0, 2, 256, 64, None) == 0
    assert lib.dg_moe_combine_backward(P(FAKE), P(FAKE), P(FAKE), None, None, P(FAKE), None, 0, 2, 256, 64, None) == 0


def test_binding_refuses_wrong_tensors():
    """The binding checks types, shapes and devices before the library is called."""
    i = torch.zeros((4, 2), dtype=torch.int32)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dg.dg_moe_sort_masked(i.long(), 8, 16, i, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError):
        dg.dg_moe_sort_masked(i, 8, 16, i, torch.zeros(8, dtype=torch.int32))          # host tensors
    with pytest.raises(TypeError):
        dg.dg_moe_dispatch_bf16(x.float(), i, None, x)
    with pytest.raises(ValueError):
        dg.dg_moe_combine(x, i, None, None, x)                                          # host tensors
    with pytest.raises(ValueError):
        dg.dg_moe_sort_contiguous(i.reshape(-1), 8, i, i.reshape(-1), i.reshape(-1))    # ids must be [T, topk]


@pytest.mark.parametrize("T", [1 << 26, 1 << 28])
def test_more_tokens_than_one_launch_holds(T):
    """A launch has fewer than 2^32 work items: one wave a token and piece (combine's gradient: four waves a token)."""
    f = P(FAKE)
    assert lib.dg_moe_dispatch_bf16(f, f, None, f, T, 1, 256, 8, None) == UNSUPPORTED
    assert lib.dg_moe_dispatch_fp8(f, f, None, f, f, T, 1, 256, 256, 128, 0, None) == UNSUPPORTED
    assert lib.dg_moe_combine(f, f, None, None, f, T, 1, 256, 8, None) == UNSUPPORTED
    assert lib.dg_moe_combine_backward(f, f, f, None, None, f, f, T >> 2, 1, 256, 8, None) == UNSUPPORTED


def test_rows_of_m_indices_count_to_the_launch():
    """... and the padding rows' waves, 16 rows each, with every row count an int holds."""
    f = P(FAKE)
    R = (1 << 31) - 128
    assert lib.dg_moe_dispatch_bf16(f, f, f, f, 0, 1, R, 8, None) == UNSUPPORTED
    assert lib.dg_moe_dispatch_bf16(f, f, f, f, 0, 1, (1 << 31) - 1, 8, None) == UNSUPPORTED
    assert lib.dg_moe_combine_backward(f, f, f, None, f, f, f, 0, 1, (1 << 31) - 1, 8, None) == UNSUPPORTED
