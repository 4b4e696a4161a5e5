"""K-grouped products whose groups, or splits of one, have no K block at all (the first one, the last one, every one),
in the tile structures that request a tile's first K blocks ahead: D = C, or zeros, and the other groups' values."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import check

pytestmark = pytest.mark.gpu
SPLIT_REFILL = ["128,128,2,2,2,1,1,6", "256,256,4,2,2,1,1,6", "128,128,2,2,3,1,1,6", "128,128,2,2,2,4,1,6"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("forced", SPLIT_REFILL + ["64,64,2,2,4,3,1,0"])
@pytest.mark.parametrize("ks,M,N", [([0, 256, 0], 264, 520), ([0, 0, 128], 130, 515), ([128, 0, 0], 512, 264), ([0, 0], 136, 136)])
def test_bf16(monkeypatch, forced, ks, M, N):
    monkeypatch.setenv("DG_FORCE_CONFIG", forced)
    K = sum(ks)
    A, B = _bf((K, M), 1), _bf((K, N), 2)
    C = torch.randn((len(ks), M, N), generator=torch.Generator().manual_seed(3))
    for c in (None, C):
        D = torch.full((len(ks), M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(A.cuda(), B.cuda(), torch.tensor(ks, dtype=torch.int32).cuda(),
                                                None if c is None else c.cuda(), D)
        at = 0
        for g, k in enumerate(ks):
            want = A[at:at + k].double().numpy().T @ B[at:at + k].double().numpy() + (0 if c is None else c[g].double().numpy())
            check.assert_close(check.bf16_to_f64(D[g].cpu()), want, f"{forced} {ks} {g}")
            at += k


@pytest.mark.parametrize("forced", SPLIT_REFILL[:3])
@pytest.mark.parametrize("M,N", [(136, 264), (40, 515)])
def test_bf16_without_any_row(monkeypatch, forced, M, N):
    monkeypatch.setenv("DG_FORCE_CONFIG", forced)
    e = lambda n: torch.empty((0, n), dtype=torch.bfloat16, device="cuda")
    C = torch.randn((M, N), device="cuda")
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_gemm_tn(e(M), e(N), None, D)
    assert not D.float().abs().sum()
    dg.dg_bf16_gemm_tn(e(M), e(N), C, D)
    assert torch.equal(D, C.to(torch.bfloat16))


@pytest.mark.parametrize("forced", [None, "128,128,2,2,2,1,1,6", "192,256,4,2,2,1,1,6"])
def test_fp8(monkeypatch, forced):
    """Codes and scales of whole numbers: every sum is exact in FP32."""
    if forced:
        monkeypatch.setenv("DG_FORCE_CONFIG", forced)
    ks, M, N = [0, 256, 0, 128, 0], 200, 264
    K = sum(ks)
    g = torch.Generator().manual_seed(1)
    A, B = (torch.randint(-4, 5, (K, n), generator=g).to(torch.float8_e4m3fn) for n in (M, N))
    sa, sb = (2.0 ** torch.randint(-1, 2, (K // 128, n), generator=g).float() for n in (M, N))
    D = torch.full((len(ks), M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_k_grouped_fp8_gemm_tn_contiguous(A.cuda(), sa.cuda(), B.cuda(), sb.cuda(),
                                           torch.tensor(ks, dtype=torch.int32).cuda(), None, D)
    a = A.double() * sa.double().repeat_interleave(128, 0)
    b = B.double() * sb.double().repeat_interleave(128, 0)
    at = 0
    for i, k in enumerate(ks):
        want = (a[at:at + k].T @ b[at:at + k]).float().to(torch.bfloat16)
        assert torch.equal(D[i].cpu(), want), i
        at += k
