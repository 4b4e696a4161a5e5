"""Argument checks of the low-rank adapters on the CPU: refused before any HIP call; their kernels' names."""
import ctypes
import glob
import os
import re
import subprocess

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd.dg import _Epilogue, _Lora, lib
from tests.test_jit import PRECOMPILE, READELF, _notes, _run
from tests.test_jit_epilogue import ACT, ALL, BF16

FAKE = 0x100000   # a 16-byte aligned address that is never dereferenced
P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(d=None), INVALID), (dict(down=None), INVALID),
    (dict(up=None), INVALID), (dict(adapter=None), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(L=0), INVALID), (dict(R=0), INVALID), (dict(act=9), INVALID), (dict(K=96), UNSUPPORTED),
    (dict(R=12), UNSUPPORTED), (dict(R=264), UNSUPPORTED), (dict(M=(1 << 24) + 1), UNSUPPORTED), (dict(N=1 << 27, R=16), UNSUPPORTED),
    (dict(a=FAKE + 8), ALIGNMENT), (dict(down=FAKE + 8), ALIGNMENT), (dict(up=FAKE + 2), ALIGNMENT),
    (dict(adapter=FAKE + 2), ALIGNMENT), (dict(scale=FAKE + 1), ALIGNMENT), (dict(bias=FAKE + 4), ALIGNMENT)])
def test_lora_refusals(kw, status):
    a = dict(a=FAKE, b=FAKE, down=FAKE, up=FAKE, adapter=FAKE, scale=FAKE, d=FAKE, bias=FAKE, act=2, M=16, N=64, K=128, L=4,
             R=16) | kw
    l = _Lora(a["down"], a["up"], a["adapter"], a["scale"], a["L"], a["R"])
    e = _Epilogue(a["bias"], 0, a["act"], None, None)
    assert lib.dg_bf16_gemm_nt_lora(P(a["a"]), P(a["b"]), ctypes.byref(l), ctypes.byref(e), P(a["d"]), a["M"], a["N"], a["K"],
                                    None) == status
    assert lib.dg_last_error().decode()


def test_lora_null_and_nothing():
    f, l = P(FAKE), _Lora(FAKE, FAKE, None, None, 4, 16)
    assert lib.dg_bf16_gemm_nt_lora(f, f, None, None, f, 16, 64, 128, None) == INVALID
    assert lib.dg_bf16_gemm_nt_lora(None, f, ctypes.byref(l), None, None, 0, 64, 128, None) == 0       # no rows


def test_lora_binding_refuses_wrong_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dg.dg_bf16_gemm_nt_lora(bf(4, 64), bf(8, 64), bf(2, 8, 64), bf(2, 8, 8), i, bf(4, 8))           # host tensors
    with pytest.raises(ValueError):
        dg.dg_bf16_gemm_nt_lora(bf(4, 64), bf(8, 64), bf(8, 64), bf(2, 8, 8), i, bf(4, 8))


@pytest.mark.parametrize("M,N,K", [(1, 512, 128), (32, 640, 256), (4096, 2048, 512)])
def test_lora_kernels_compile_ahead(M, N, K):
    """dg_describe_config names them and dg_precompile compiles them (no GPU); other forms have none."""
    kind = dg.KIND_BF16 | dg.EPI_LORA
    assert dg.describe_config(kind, M, N, K, 1, 0, 256).endswith("_lora")
    dg.precompile(kind, M, N, K, 1, 0, 256)
    for other in (dg.EPI_LORA, kind | 1, kind | 2, kind | 3, kind | dg.LAYOUT_NN):
        with pytest.raises(dg.DGError):
            dg.describe_config(other, 128, N, 128, 1, 0, 256)


@pytest.mark.skipif(not os.path.exists(READELF), reason="LLVM tools not installed")
def test_lora_kernels_compile_without_scratch(tmp_path):
    """On every tile structure, with no other part of the epilogue and with all of them; the kernel's argument ends
    with the adapters."""
    kind, full = BF16 | dg.EPI_LORA, ALL | ACT["gelu"]
    shapes = {"256n256": (4096, 7168, 2048), "128n256": (3000, 2111, 1024), "128n192": (2560, 7001, 64),
              "192n128": (2049, 8000, 64), "128n128": (2049, 2111, 64), "128n64": (517, 2112, 1536), "64n128": (1000, 2111, 64),
              "64n64": (1000, 1100, 64), "32n64": (600, 768, 256), "32n32": (32, 7168, 2048), "16n32": (16, 640, 256)}
    plans = [(kind | extra, *s, 1, 0) for s in shapes.values() for extra in (0, full)]
    for tile, s in shapes.items():
        assert f"_m{tile}_" in dg.describe_config(kind, *s, 1, 0, 256)
    r = _run(PRECOMPILE.format(plans=repr(plans)), tmp_path)
    assert r.returncode == 0, r.stderr[-2000:]
    assert all(line.split(")")[1].split()[0] == "0" for line in r.stdout.strip().splitlines()), r.stdout
    objs = glob.glob(str(tmp_path / "*.hsaco"))
    assert len(objs) == len(plans)
    for path in objs:
        name, v = os.path.basename(path), _notes(path)
        assert not max(v["vgpr_spill_count"]) and not max(v["private_segment_fixed_size"]), (name, v)
        out = subprocess.run([READELF, "--notes", path], capture_output=True, text=True).stdout
        assert re.search(r"\.size:\s+152\s+\.value_kind:\s+by_value", out), name
