"""Arrays of more than 2^32 elements: the rows at their ends come out as they do alone, bit for bit."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg

pytestmark = pytest.mark.gpu
ENDS = 200


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _rows(T, H, dtype=torch.bfloat16):
    """[T,H], zeros but for the ENDS first and last rows; and those two."""
    x = torch.zeros((T, H), dtype=dtype, device="cuda")
    x[:ENDS].normal_()
    x[-ENDS:].normal_()
    return x, (x[:ENDS].clone(), x[-ENDS:].clone())


def _ends(t):
    return t[:ENDS], t[-ENDS:]


def test_norm():
    T, H = 600001, 7168
    x, ends = _rows(T, H)
    y = torch.empty_like(x)
    q, sf = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((H // 128, T), device="cuda")
    dg.dg_rms_norm(x, None, 1e-5, Y=y, Q=q, sf=sf)
    for e, gy, gq, gs in zip(ends, _ends(y), _ends(q), _ends(sf.t())):
        y1, q1, s1 = torch.empty_like(e), torch.empty_like(e, dtype=torch.uint8), torch.empty((H // 128, ENDS), device="cuda")
        dg.dg_rms_norm(e, None, 1e-5, Y=y1, Q=q1, sf=s1)
        assert torch.equal(gy, y1) and torch.equal(gq, q1) and torch.equal(gs, s1.t())
    dg.dg_rms_norm_backward(x, x, None, 1e-5, y, None)
    for e, g in zip(ends, _ends(y)):
        y1 = torch.empty_like(e)
        dg.dg_rms_norm_backward(e, e, None, 1e-5, y1, None)
        assert torch.equal(g, y1)


def test_route():
    T, E, k = (1 << 22) + 77, 1024, 4
    l, ends = _rows(T, E)
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    dg.dg_moe_route(l, None, ids, w)
    d = torch.empty_like(l)
    dg.dg_moe_route_backward(l, ids, w, d)
    for e, gi, gw, gd in zip(ends, _ends(ids), _ends(w), _ends(d)):
        i1, w1, d1 = torch.empty_like(gi), torch.empty_like(gw), torch.empty_like(e)
        dg.dg_moe_route(e, None, i1, w1)
        dg.dg_moe_route_backward(e, i1, w1, d1)
        assert torch.equal(gi, i1) and torch.equal(gw, w1) and torch.equal(gd, d1)


def test_checkpoint():
    M, N = (1 << 20) + 77, 4100
    x, ends = _rows(M, N)
    codes = torch.empty((M, N), dtype=torch.uint8, device="cuda")
    scales = torch.empty((M, 33), dtype=torch.uint8, device="cuda")
    dg.dg_checkpoint_fp8(x, codes, scales)
    back, h = torch.empty_like(x), torch.empty_like(x)
    dg.dg_checkpoint_restore(codes, scales, back)
    dz = torch.empty_like(x)
    dg.dg_epilogue_backward_fp8(x, codes, scales, "silu", dz, None, H=h)
    for e, gc, gs, gb, gz, gh in zip(ends, _ends(codes), _ends(scales), _ends(back), _ends(dz), _ends(h)):
        c1, s1 = torch.empty_like(gc), torch.empty_like(gs)
        b1, z1, h1 = torch.empty_like(e), torch.empty_like(e), torch.empty_like(e)
        dg.dg_checkpoint_fp8(e, c1, s1)
        dg.dg_checkpoint_restore(c1, s1, b1)
        dg.dg_epilogue_backward_fp8(e, c1, s1, "silu", z1, None, H=h1)
        for got, want in ((gc, c1), (gs, s1), (gb, b1), (gz, z1), (gh, h1)):
            assert torch.equal(got, want)


def test_low_rank_adapters():
    """The last of 17 adapters whose factors are 2^28 elements each."""
    L, R, N, K, M = 17, 256, 1 << 20, 64, 33
    up, down = torch.zeros((L, N, R), dtype=torch.bfloat16, device="cuda"), torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    up[L - 1].normal_()
    down[L - 1].normal_()
    A, B = torch.randn((M, K), device="cuda").bfloat16(), torch.randn((N, K), device="cuda").bfloat16()
    D, D1 = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.full((M,), L - 1, dtype=torch.int32, device="cuda")
    dg.dg_bf16_gemm_nt_lora(A, B, down, up, ids, D)
    dg.dg_bf16_gemm_nt_lora(A, B, down[L - 1:].contiguous(), up[L - 1:].contiguous(), ids * 0, D1)
    assert torch.equal(D, D1)
    dg.dg_bf16_gemm_nt_lora(A, B, down, up, ids - 1, D1)
    assert not torch.equal(D, D1)
