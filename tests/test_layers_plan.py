"""Which kernels the layer operators' host code chooses and what it lays out for
them, without a GPU: its launchers are replaced by a record of their arguments."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "sparsified_gradient_compression_amd", "csrc")


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_what_is_launched(tmp_path):
    exe = str(tmp_path / "layers_plan_check")
    r = subprocess.run(["hipcc", "--offload-arch=gfx950", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                        os.path.join(CSRC, "dgc_layers.hip"), os.path.join(ROOT, "tests", "layers_plan_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "plan check: ok" in r.stdout, r.stderr
