"""DG_FORCE_CONFIG: a configuration that its kernel is not built and tested for is not taken, the call's own choice is."""
import pytest

import moe_grouped_gemm_scales_amd as dg


def _key(kind, N=512, K=2048):
    return dg.describe_config(kind, 128, N, K, 1 if kind & 3 == 0 else 4, num_cus=256)


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("variant", [1, 2, 3, 4, 5])
def test_split_k_of_grouped_forms_is_for_variants_0_and_6(monkeypatch, kind, variant):
    tile = {1: "64,64,1,4,4,2,1,1", 2: "32,64,1,4,4,2,1,2", 3: "64,96,1,6,3,2,1,3", 4: "128,128,4,2,2,2,1,4",
            5: "128,256,1,8,4,2,1,5"}[variant]
    own = _key(kind)
    monkeypatch.setenv("DG_FORCE_CONFIG", tile)
    assert _key(kind) == own
    monkeypatch.setenv("DG_FORCE_CONFIG", tile.replace(",2,1,%d" % variant, ",1,1,%d" % variant))   # unsplit: taken
    assert _key(kind).startswith(f"k{kind}v{variant}_")


@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("tile", ["64,64,2,2,4,2,1,0", "128,128,2,2,2,2,1,6"])
def test_split_k_of_grouped_forms(monkeypatch, kind, tile):
    monkeypatch.setenv("DG_FORCE_CONFIG", tile)
    assert "x1_sk2_" in _key(kind)


@pytest.mark.parametrize("tile", ["64,64,1,4,4,2,1,1", "32,64,1,4,4,2,1,2", "64,96,1,6,3,2,1,3"])
def test_split_k_of_the_dense_form_is_for_more_variants(monkeypatch, tile):
    monkeypatch.setenv("DG_FORCE_CONFIG", tile)
    assert f"k0v{tile[-1]}_" in _key(0) and "x1_sk2_" in _key(0)
