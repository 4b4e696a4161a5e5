"""The package without its tensor-check extension: it imports, the calls that never used the extension and those that
do are there, and refuse the same arguments with the same errors."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd import dg as binding

PKG = os.path.dirname(os.path.abspath(dg.__file__))
CHECK = """
import torch
import moe_grouped_gemm_scales_amd as dg
from moe_grouped_gemm_scales_amd import dg as binding
assert binding._pycheck is None and dg.__file__.startswith({root!r}), dg.__file__
assert dg.describe_config(0, 64, 256, 256, num_cus=256)
a, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
i = torch.zeros((4, 2), dtype=torch.int32)
for call, error in [(lambda: dg.dg_bf16_gemm_nt_epilogue(a.float(), w, a), TypeError),
                    (lambda: dg.dg_bf16_gemm_nt_epilogue(a, w, a), ValueError),
                    (lambda: dg.dg_moe_sort_masked(i.long(), 8, 16, i, i), TypeError),
                    (lambda: dg.dg_moe_combine(a, i, None, None, a), ValueError),
                    (lambda: dg.dg_bf16_gemm_nt(a, w, None, a), ValueError)]:
    try:
        call()
    except error:
        continue
    raise SystemExit("not refused")
print("imported")
"""


@pytest.mark.parametrize("extension", ["absent", "not a library", "of another torch"])
def test_import_without_the_extension(tmp_path, extension):
    root = tmp_path / "moe_grouped_gemm_scales_amd"
    root.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py"):
            shutil.copy(os.path.join(PKG, name), root / name)
    os.symlink(os.path.join(PKG, "libdg.so"), root / "libdg.so")
    if extension == "not a library":
        (root / "_pycheck.so").write_bytes(b"no library")
    if extension == "of another torch":
        # the built one, with the version in it overwritten by as many bytes
        v = torch.__version__.split("+")[0].encode()
        data = open(os.path.join(PKG, "_pycheck.so"), "rb").read()
        assert v + b"\0" in data
        (root / "_pycheck.so").write_bytes(data.replace(v + b"\0", b"0" * len(v) + b"\0"))
    r = subprocess.run([sys.executable, "-c", CHECK.format(root=str(root))], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)}, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stdout + r.stderr


def _outcome(f, *args):
    try:
        return f(*args)
    except Exception as e:
        return type(e), str(e)


def _compare(t, dev):
    """Both checks of one tensor against several wishes, each met or refused in the same way."""
    for other in (t, t.float(), t[:, 1:], t.t(), t[:0], t.cpu(), None, 3, [1]):
        for dtype in (torch.bfloat16, torch.float32):
            for shape in ((4, 6), (4, 5), (6, 4), (0, 6), (24,)):
                args = (other, "t", dtype, shape, dev)
                assert _outcome(binding._arg, *args) == _outcome(binding._arg_in_python, *args), args
                assert _outcome(binding._opt, *args) == _outcome(binding._opt_in_python, *args), args


def test_both_checks_agree_on_host_tensors(monkeypatch):
    assert binding._pycheck is not None
    monkeypatch.setattr(binding, "_cur_device", lambda: 0)
    _compare(torch.zeros((4, 6), dtype=torch.bfloat16), 0)


@pytest.mark.gpu
def test_both_checks_agree_on_device_tensors():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _compare(torch.zeros((4, 6), dtype=torch.bfloat16, device="cuda"), torch.cuda.current_device())
