"""Contiguous form in 256-row tiles over an odd number of 128-row blocks: the last tile is half past the rows, and
past m_indices.  Its rows, and only they, are computed, in wave tiles that find each row's expert in memory as well as
in those that bring the experts into LDS."""
import pytest
import torch

from tests import check, gen, gpu_util

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()


@pytest.mark.parametrize("forced", ["256,128,2,4,2,1,1,0", "256,64,2,2,2,1,1,0", "256,256,4,2,2,1,1,6"])
@pytest.mark.parametrize("rows,pad", [([128], 0), ([200, 100, 0, 250], 0), ([384, 1], 128)])
@pytest.mark.parametrize("bf16", [True, False])
def test_odd_number_of_row_blocks(monkeypatch, oracle, forced, rows, pad, bf16):
    monkeypatch.setenv("DG_FORCE_CONFIG", forced)
    N, K = 264, 512
    p = gen.make_bf16("contiguous", seed=3, N=N, K=K, group_rows=rows, pad_rows=pad) if bf16 else \
        gen.make_contiguous(rows, N, K, seed=3, pad_rows=pad)
    assert len(p.m_indices) % 256 == 128, len(p.m_indices)
    D, sent = gpu_util.run(p)
    want, computed = gpu_util.oracle_rows(oracle, p)
    check.assert_close(check.bf16_to_f64(D)[computed], want[computed], forced)
    assert torch.equal(D[torch.from_numpy(~computed)].view(torch.int16), sent[torch.from_numpy(~computed)].view(torch.int16))
