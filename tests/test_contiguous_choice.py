"""Tile structures of contiguous products with a fused epilogue, and of the NN form, over many rows: 256 x 256 where its
whole rounds outweigh the tiles that two experts share, 128 x 256 where there are many experts or few rounds.  The
sides of each choice were measured apart by 6 % or more."""
import pytest

import moe_grouped_gemm_scales_amd as dg

EPI = 1 | dg.EPI_BIAS_F32 | (dg.ACTIVATIONS["silu"] << 12)


def _tile(kind, M, N, K, G):
    return dg.describe_config(kind, M, N, K, G, num_cus=256).split("_")[1]


@pytest.mark.parametrize("M,N,K,G,tile", [
    (32768, 4096, 7168, 4, "m256n256"), (32768, 4096, 7168, 8, "m256n256"), (65536, 4096, 7168, 4, "m256n256"),
    (32768, 7168, 2048, 4, "m256n256"), (8192, 4096, 7168, 4, "m128n256"), (8192, 4096, 7168, 32, "m128n256"),
    (16384, 4096, 7168, 32, "m128n256"), (8192, 7168, 2048, 16, "m128n256")])
def test_fp8(M, N, K, G, tile):
    assert _tile(EPI, M, N, K, G) == tile


@pytest.mark.parametrize("M,N,K,G,tile", [
    (32768, 4096, 4096, 4, "m256n256"), (65536, 4096, 4096, 8, "m256n256"), (32768, 7168, 2048, 4, "m256n256"),
    (32768, 4096, 4096, 32, "m128n256"), (32768, 2048, 4096, 16, "m128n256"), (8192, 4096, 4096, 4, "m128n256"),
    (16384, 4096, 4096, 32, "m128n256")])
@pytest.mark.parametrize("kind", [EPI | dg.KIND_BF16, 1 | dg.KIND_BF16 | dg.LAYOUT_NN])
def test_bf16(kind, M, N, K, G, tile):
    assert _tile(kind, M, N, K, G) == tile
