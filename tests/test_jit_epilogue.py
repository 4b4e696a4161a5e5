"""The hipRTC build, on the CPU, of the products with a fused epilogue and of the BF16 K-grouped product:
every part of the epilogue compiles for gfx950 without scratch memory, and the kernel's one argument grows
by the epilogue's three pointers."""
import glob
import os
import re
import subprocess

import pytest

from tests.test_jit import PRECOMPILE, READELF, _k_loop_scratch_ops, _notes, _run

BF16, BIAS, BIAS16, RES, Z = 16, 0x100, 0x200, 0x400, 0x800
ACT = {"relu": 1 << 12, "silu": 2 << 12, "gelu": 3 << 12, "gelu_tanh": 4 << 12}
ALL = BIAS | RES | Z

PLANS = [
    # large tiles (256 x 256), every part at once
    (0 | BF16 | ALL | ACT["gelu"], 4096, 7168, 4096, 1, 0), (0 | ALL | ACT["gelu_tanh"], 4096, 7168, 16384, 1, 0),
    (1 | ALL | ACT["gelu"], 32768, 4096, 7168, 4, 0), (1 | BF16 | ALL | ACT["gelu"], 32768, 4096, 7168, 4, 0),
    # few rows: split-K, the variants that load B into registers
    (0 | BF16 | BIAS16 | ACT["silu"], 1, 7168, 2048, 1, 0), (0 | ALL | ACT["silu"], 64, 2112, 7168, 1, 0),
    (0 | ALL | ACT["relu"], 128, 24576, 1536, 1, 0), (2 | ALL | ACT["gelu"], 256, 7168, 2048, 4, 0),
    (2 | BF16 | ALL | ACT["gelu"], 256, 7168, 2048, 4, 0),
    # odd widths: 8-byte and single stores
    (0 | BF16 | ALL | ACT["gelu"], 517, 2116, 1536, 1, 0), (0 | BF16 | ALL | ACT["gelu_tanh"], 300, 515, 640, 1, 0),
    # the BF16 K-grouped product
    (3 | BF16, 4096, 7168, 8192, 4, 0), (3 | BF16, 2112, 1536, 1500, 1, 0), (3 | BF16, 40, 72, 128, 3, 1),
]


@pytest.mark.skipif(not os.path.exists(READELF), reason="LLVM tools not installed")
def test_epilogue_kernels_compile_without_scratch(tmp_path):
    r = _run(PRECOMPILE.format(plans=repr(PLANS)), tmp_path)
    assert r.returncode == 0, r.stderr[-2000:]
    assert all(line.split(")")[1].split()[0] == "0" for line in r.stdout.strip().splitlines()), r.stdout
    objs = glob.glob(str(tmp_path / "*.hsaco"))
    assert len(objs) >= len(PLANS)
    for path in objs:
        name, v = os.path.basename(path), _notes(path)
        assert not _k_loop_scratch_ops(path), f"{name}: scratch access in the K loop"
        assert not max(v["vgpr_spill_count"]) and not max(v["private_segment_fixed_size"]), (name, v)
        out = subprocess.run([READELF, "--notes", path], capture_output=True, text=True).stdout
        assert re.search(r"\.size:\s+%d\s+\.value_kind:\s+by_value" % (120 if "_ep" in name else 96), out), name


def test_unknown_activation_is_refused():
    import moe_grouped_gemm_scales_amd as dg
    with pytest.raises(dg.DGError):
        dg.precompile(0 | BF16 | (5 << 12), 64, 64, 64, num_cus=256)
    key = dg.describe_config(0 | dg.KIND_BF16 | dg.EPI_BIAS_F32 | dg.EPI_Z | ACT["gelu"], 64, 512, 512, num_cus=256)
    assert key.endswith("_ep1301")


def test_every_structure_is_chosen_somewhere():
    """Shapes over the whole range reach each of the tile structures."""
    import itertools

    import moe_grouped_gemm_scales_amd as dg
    seen = set()
    for kind, fp8 in itertools.product((0, 1, 2), (False, True)):
        for M, N, K in itertools.product((1, 16, 24, 64, 200, 517, 1024, 3000, 8192, 32768), (520, 2112, 4096, 7168), (1536, 7168)):
            if kind == 1:
                M = (M + 127) // 128 * 128
            key = dg.describe_config(kind | (0 if fp8 else BF16) | BIAS, M, N, K, 1 if kind == 0 else 4, num_cus=256)
            seen.add(re.search(r"_m(\d+n\d+)_", key).group(1))
    want = {"256n256", "128n256", "128n192", "192n128", "128n128", "128n64", "64n128", "64n64", "32n64", "16n64", "16n32"}
    assert want <= seen, want - seen
