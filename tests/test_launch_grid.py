"""Launches next to HIP's limit of 2^32 threads along x, which some thousand
million gradients or rows reach: the grids, on the host."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "sparsified_gradient_compression_amd", "csrc")


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_grids_on_either_side_of_the_limit(tmp_path):
    exe = str(tmp_path / "grid_check")
    r = subprocess.run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-I", CSRC,
                        os.path.join(ROOT, "tests", "launch_grid_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "grid check: ok" in r.stdout, r.stderr
