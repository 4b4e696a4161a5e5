"""How many kernels a TN product needs over a range of token counts, and that a few calls meet them all: the same plan
within an eighth of an octave of K."""
import pytest

import moe_grouped_gemm_scales_amd as dg

TN = 3 | dg.KIND_BF16


def _key(M, N, K, G=1):
    return dg.describe_config(TN, M, N, K, G, num_cus=256)


@pytest.mark.parametrize("M,N,G,kernels", [(512, 512, 1, 5), (4096, 7168, 1, 2), (4096, 2048, 8, 1)])
def test_kernels_over_token_counts(M, N, G, kernels):
    assert len({_key(M, N, K, G) for K in range(128, 32769, 128)}) == kernels


@pytest.mark.parametrize("M,N", [(512, 512), (192, 200), (1600, 1408)])
def test_one_call_of_each_range_meets_every_plan(M, N):
    """K blocks of 64, the ranges of equal leading four bits: b, b + b // 8, ..."""
    met, b = set(), 1
    while b <= 512:
        met.add(_key(M, N, 64 * b))
        b += max(1, (1 << (b.bit_length() - 1)) // 8)
    assert {_key(M, N, K) for K in range(1, 32769, 61)} <= met
