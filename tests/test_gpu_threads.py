"""Host threads that queue calls on one stream: what a call's first kernel hands to its second (a sort's
counts, the partial sums of a bias gradient) must not be another call's."""
import threading

import numpy as np
import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from tests import moe_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


def _sorter(seed, calls):
    """Sorts of one set of ids, each into its own places."""
    T, k, G = 6000, 4, 24 + seed
    ids = np.random.default_rng(seed).integers(0, G, (T, k)).astype(np.int32)
    rows = dg.moe_sorted_rows(T, k, G)
    d_ids = torch.from_numpy(ids).cuda()
    out = [[torch.empty(n, dtype=torch.int32, device="cuda") for n in ((T, k), (rows,), (G,))] for _ in range(calls)]

    def run():
        for o in out:
            dg.dg_moe_sort_contiguous(d_ids, G, *o)

    def check():
        want = ref.sort_contiguous(ids, G, rows)
        for o in out:
            for got, w in zip(o, want):
                assert np.array_equal(got.cpu().numpy(), w)
    return run, check


def _bias(seed, calls):
    """Bias gradients of whole numbers (their sums are exact in any order)."""
    M, N = 1024, 512 + 64 * seed
    dD = torch.from_numpy(np.random.default_rng(seed).integers(-8, 9, (M, N)).astype(np.float32)).to(torch.bfloat16)
    d = dD.cuda()
    out = [torch.empty(N, device="cuda") for _ in range(calls)]

    def run():
        for o in out:
            dg.dg_epilogue_backward(d, None, "none", None, o)

    def check():
        want = dD.double().sum(0)
        for o in out:
            assert torch.equal(o.cpu().double(), want)
    return run, check


def _split_k(seed, calls):
    """Products of few rows over a long K: their splits' partial sums use the stream's workspace too."""
    A, B = torch.ones((16, 7168), dtype=torch.bfloat16, device="cuda"), torch.ones((2112, 7168), dtype=torch.bfloat16, device="cuda")
    out = [torch.empty((16, 2112), dtype=torch.bfloat16, device="cuda") for _ in range(calls)]

    def run():
        for o in out:
            dg.dg_bf16_gemm_nt_epilogue(A, B, o)

    def check():
        for o in out:
            assert bool((o == 7168).all())
    return run, check


def test_threads_share_a_stream():
    work = [make(seed, 60) for seed, make in enumerate((_sorter, _sorter, _bias, _bias, _split_k))]
    for run, _ in work:           # compiled, allocated and warm before the threads start
        run()
    torch.cuda.synchronize()
    start = threading.Barrier(len(work))
    failed = []

    def body(run):
        try:
            start.wait(60)
            for _ in range(5):
                run()
        except Exception as e:     # reported by the main thread
            failed.append(e)

    threads = [threading.Thread(target=body, args=(run,)) for run, _ in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join(100)
    assert not failed and not any(t.is_alive() for t in threads)
    torch.cuda.synchronize()
    for _, check in work:
        check()
