"""Which kernel a call takes does not depend on which calls came before it: two products of the same sizes whose
choices differ (the plain BF16 NT form, and the NN form whose B is rewritten first) keep their own plans."""
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg

pytestmark = pytest.mark.gpu
M, K = 300, 1024
NT, NN = 0 | dg.KIND_BF16, 0 | dg.KIND_BF16 | dg.LAYOUT_NN


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


@pytest.mark.parametrize("first,N", [("nt", 515), ("nn", 517)])
def test_plans_of_both_forms(monkeypatch, capfd, first, N):
    keys = {"nt": dg.describe_config(NT, M, N, K), "nn": dg.describe_config(NN, M, N, K)}
    assert keys["nt"] != keys["nn"]          # the sizes of this test
    a = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    b = torch.ones((N, K), dtype=torch.bfloat16, device="cuda")
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    calls = {"nt": lambda: dg.dg_bf16_gemm_nt(a, b, None, d), "nn": lambda: dg.dg_bf16_gemm_nn(a, b.reshape(K, N), None, d)}
    monkeypatch.setenv("DG_PRINT_CONFIGS", "1")
    capfd.readouterr()
    for form in (first, "nn" if first == "nt" else "nt", first):
        d.zero_()
        calls[form]()
        torch.cuda.synchronize()
        launched = [line.split()[2] for line in capfd.readouterr().err.splitlines() if line.startswith("[dg] launch")]
        assert launched == [keys[form]], form
        assert bool((d == K).all())
