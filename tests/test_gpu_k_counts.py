"""K-grouped counts whose sum passes 31 bits: the segments are cut at K like any that exceed it, negative counts are 0."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg

pytestmark = pytest.mark.gpu
BIG = 2 ** 31 - 128
K = 640


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _segments(ks):
    at, out = 0, []
    for k in ks:
        n = min(max(k, 0), K - at)
        out.append(slice(at, at + n))
        at += n
    return out


@pytest.mark.parametrize("form", ["bf16 as stored", "bf16 rewritten", "fp8"])
@pytest.mark.parametrize("ks", [[BIG, 128], [128, BIG, 128], [1 << 30] * 4, [256, -128, 1 << 30, 1 << 30, -BIG, BIG], [BIG] * 5,
                                [128, 2 ** 31 - 1]])
def test_counts_past_31_bits(form, ks):
    M, N = (72, 520) if form != "bf16 rewritten" else (70, 515)
    g = torch.Generator().manual_seed(1)
    ints = lambda n: torch.randint(-3, 4, (K, n), generator=g)      # sums exact in FP32
    a, b = ints(M), ints(N)
    D = torch.full((len(ks), M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    d_ks = torch.tensor(ks, dtype=torch.int32).cuda()
    if form == "fp8":
        one = lambda n: torch.ones((K // 128, n), device="cuda")
        dg.dg_k_grouped_fp8_gemm_tn_contiguous(a.to(torch.float8_e4m3fn).cuda(), one(M), b.to(torch.float8_e4m3fn).cuda(),
                                               one(N), d_ks, None, D)
    else:
        dg.dg_k_grouped_bf16_gemm_tn_contiguous(a.to(torch.bfloat16).cuda(), b.to(torch.bfloat16).cuda(), d_ks, None, D)
    for i, s in enumerate(_segments(ks)):
        want = (a[s].double().T @ b[s].double()).float().to(torch.bfloat16)
        assert torch.equal(D[i].cpu(), want), (i, s)
