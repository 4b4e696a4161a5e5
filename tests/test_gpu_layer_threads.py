"""Host threads that queue calls on one stream: a low-rank product, the partial sums of a norm's weight and those of a
bias gradient stand in the same workspace, and each call gets its own result, bit for bit that of a call alone."""
import threading

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests.test_gpu_norm import _bf

pytestmark = pytest.mark.gpu
CALLS = 60


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _lora(seed):
    M, N, K, R, L = 40 + 300 * seed, 512, 512, 16 + 16 * seed, 5
    a, b, down, up = (_bf(s, seed + i).cuda() for i, s in enumerate([(M, K), (N, K), (L, R, K), (L, N, R)]))
    ids = (torch.arange(M, dtype=torch.int32) * (1 + seed) % L).cuda()
    return torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), lambda D: dg.dg_bf16_gemm_nt_lora(a, b, down, up, ids, D)


def _norm(seed):
    dy, s = _bf((900, 1000), 20 + seed).cuda(), _bf((900, 1000), 30 + seed).cuda()
    return torch.empty(1000, device="cuda"), lambda dw: dg.dg_rms_norm_backward(dy, s, None, 1e-5, None, dw)


def _kept(seed):
    dd, z = _bf((1024, 640), 40 + seed).cuda(), _bf((1024, 640), 50 + seed).cuda()
    codes, scales = torch.empty((1024, 640), dtype=torch.uint8, device="cuda"), torch.empty((1024, 5), dtype=torch.uint8, device="cuda")
    dg.dg_checkpoint_fp8(z, codes, scales)
    return torch.empty(640, device="cuda"), lambda db: dg.dg_epilogue_backward_fp8(dd, codes, scales, "silu", None, db)


def test_threads_on_one_stream():
    work = [make(seed) for make in (_lora, _norm, _kept) for seed in (0, 1)]
    want = []
    for out, call in work:
        call(out)
        want.append(out.clone())
    got = [[torch.empty_like(out) for _ in range(CALLS)] for out, _ in work]
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            for o in got[i]:
                work[i][1](o)
        except Exception as e:          # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for w, outs in zip(want, got):
        for o in outs:
            assert torch.equal(o, w)
