"""The sort at the largest row count it takes: 2^31 - 128, whose last indices lie within one step of 2^31."""
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


def test_sort_into_the_most_rows():
    T, k, G = 100000, 3, 5
    ids = np.random.default_rng(1).integers(-1, G, (T, k)).astype(np.int32)
    R = (1 << 31) - 128
    pos = torch.empty((T, k), dtype=torch.int32, device="cuda")
    ks = torch.empty(G, dtype=torch.int32, device="cuda")
    buf = torch.full((R + 4096,), 77, dtype=torch.int32, device="cuda")
    dg.dg_moe_sort_contiguous(torch.from_numpy(ids).cuda(), G, pos, buf[:R], ks)
    n = ref.sorted_rows(T, k, G)
    wp, wm, wk = ref.sort_contiguous(ids, G, n)
    assert np.array_equal(pos.cpu().numpy(), wp) and np.array_equal(ks.cpu().numpy(), wk)
    assert np.array_equal(buf[:n].cpu().numpy(), wm)
    for at in range(n, R, 1 << 28):
        assert bool((buf[at:min(at + (1 << 28), R)] == -2).all()), at
    assert bool((buf[R:] == 77).all())
