"""Device code of the plaintext-side kernels as host code (no GPU): threads are
fibers, barriers and moves between lanes are emulated (tests/native/hip/
hip_runtime.h stands in for the runtime's header)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = next((c for c in ("/opt/rocm/llvm/bin/clang++", "clang++") if shutil.which(c)), None)  # vector types


def _run(tmp_path, source, check):
    if CLANG is None:
        pytest.skip("clang++ not available")
    path = os.path.join(ROOT, "rns_ckks_polynomial_amd", "csrc", "plain")
    with open(os.path.join(path, source)) as f:
        device, mark, _ = f.read().partition("}  // namespace ckks_plain\n")  # the launches follow
    assert mark
    (tmp_path / "sample_device.inc").write_text(device + mark)
    exe = str(tmp_path / "check")
    subprocess.run([CLANG, "-std=c++17", "-O1", "-w", "-I", os.path.join(ROOT, "tests", "native"), "-I", str(tmp_path),
                    "-I", path, "-o", exe, os.path.join(ROOT, "tests", "native", check)], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_selection_from_a_list(tmp_path):
    assert "select: ok" in _run(tmp_path, "sample.hip", "sample_select_check.cpp")
