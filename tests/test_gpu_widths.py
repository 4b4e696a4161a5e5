"""Gradients at widths that are no multiple of 64: whatever width a forward product has, its operand's gradient
dA = dZ . B, whose K is that width, follows.  Bounds as in tests/test_gpu_linear.py."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import check
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _bf(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def _poison_workspace(M, N, K):
    """A product that leaves NaN in the stream's workspace, past and inside the operands of the next one."""
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_bf16_gemm_nn(nan(M + 8, K + 131), nan(K + 131, N + 8 | 1), None, torch.empty((M + 8, N + 8 | 1), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("with_c", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 129, 7), (64, 2112, 1000), (257, 515, 65), (300, 7, 515), (517, 1536, 2139),
                                   (33, 264, 2116), (2048, 1024, 4478), (1, 4096, 100)])
def test_nn_of_any_k(M, N, K, with_c):
    A, B = _bf((M, K), 1), _bf((K, N), 2)
    C = torch.randn((M, N), generator=torch.Generator().manual_seed(3)) if with_c else None
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    _poison_workspace(M, N, K)
    dg.dg_bf16_gemm_nn(A.cuda(), B.cuda(), None if C is None else C.cuda(), D)
    want = A.double().numpy() @ B.double().numpy() + (0 if C is None else C.double().numpy())
    check.assert_close(check.bf16_to_f64(D.cpu()), want, f"nn {M}x{N}x{K}")


@pytest.mark.parametrize("K", [1, 63, 100, 515, 1000])
@pytest.mark.parametrize("N", [64, 515])
def test_contiguous_nn_of_any_k(N, K):
    m = []
    for g, c in enumerate([128, 0, 200, 100]):
        m += [g] * c + [-1] * (-c % 128)
    m = torch.tensor(m + [-2] * 128, dtype=torch.int32)
    A, B = _bf((len(m), K), 1), _bf((4, K, N), 2)
    A[m < 0] = float("nan")
    D = torch.full((len(m), N), float("inf"), dtype=torch.bfloat16, device="cuda")
    _poison_workspace(len(m), N, K)
    dg.dg_m_grouped_bf16_gemm_nn_contiguous(A.cuda(), B.cuda(), m.cuda(), None, D)
    D, keep = D.cpu(), m >= 0
    want = np.stack([A[r].double().numpy() @ B[int(m[r])].double().numpy() for r in torch.nonzero(keep)[:, 0].tolist()])
    check.assert_close(check.bf16_to_f64(D[keep]), want, "nn contiguous")
    assert torch.isinf(D[~keep].float()).all()


@pytest.mark.parametrize("N", [100, 515, 1000, 2139])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_layer_forward_and_backward(N, act):
    """Forward with Z, dZ, dbias, dA and dB of one width, each from the values that the call before it stored."""
    M, K = 150, 192
    x, w, dd = _bf((M, K), 1), _bf((N, K), 2, 0.1), _bf((M, N), 3)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(4))
    new = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    D, Z, dZ, dA, dB = new(M, N), new(M, N), new(M, N), new(M, K), new(N, K)
    db = torch.empty(N, device="cuda")
    xc, wc = x.cuda(), w.cuda()
    dg.dg_bf16_gemm_nt_epilogue(xc, wc, D, bias=bias.cuda(), activation=act, Z=Z)
    dg.dg_epilogue_backward(dd.cuda(), Z, act, dZ, db)
    dg.dg_bf16_gemm_nn(dZ, wc, None, dA)
    dg.dg_bf16_gemm_tn(dZ, xc, None, dB)
    z = x.double().numpy() @ w.double().numpy().T + bias.double().numpy()
    check.assert_close(check.bf16_to_f64(Z.cpu()), z, "Z")
    zz, d = Z.cpu().double().numpy(), dd.double().numpy()
    want = d * ref.slope(zz, act)
    slack = 2.0 ** -20 * np.abs(d) * (1 + np.abs(zz))
    assert np.all(np.abs(dZ.cpu().double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + slack)
    assert np.all(np.abs(db.cpu().double().numpy() - want.sum(0)) <= slack.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(want).sum(0))
    g = dZ.cpu().double().numpy()
    check.assert_close(check.bf16_to_f64(dA.cpu()), g @ w.double().numpy(), "dA")
    check.assert_close(check.bf16_to_f64(dB.cpu()), g.T @ x.double().numpy(), "dB")


def test_replays_from_a_graph():
    M, N, K = 200, 136, 515
    A, B = _bf((M, K), 1).cuda(), _bf((K, N), 2).cuda()
    D, E = (torch.zeros((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.dg_bf16_gemm_nn(A, B, None, D)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dg.dg_bf16_gemm_nn(A, B, None, D)
    for seed in range(4):
        A.copy_(_bf((M, K), 20 + seed))
        D.zero_()
        torch.cuda.synchronize()
        dg.dg_bf16_gemm_nn(A, B, None, E)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D.view(torch.int16), E.view(torch.int16)), seed
