"""Device code of the alternatives of token_logprobs and of the order of tokens
as host code (no GPU; tests/native/hip/hip_runtime.h stands in for the
runtime's header)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = next((c for c in ("/opt/rocm/llvm/bin/clang++", "clang++") if shutil.which(c)), None)  # vector types


def _run(tmp_path, source, check, replaced=()):
    if CLANG is None:
        pytest.skip("clang++ not available")
    path = os.path.join(ROOT, "rns_ckks_polynomial_amd", "csrc", "plain")
    with open(os.path.join(path, source)) as f:
        device, mark, _ = f.read().partition("// ------------------------------------------------------------------ launches")
    assert mark
    for a, b in replaced:
        assert a in device
        device = device.replace(a, b)
    (tmp_path / "device.inc").write_text(device + "}\n")
    exe = str(tmp_path / "check")
    subprocess.run([CLANG, "-std=c++17", "-O2", "-w", "-I", os.path.join(ROOT, "tests", "native"), "-I", str(tmp_path),
                    "-I", path, "-o", exe, os.path.join(ROOT, "tests", "native", check)], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_alternatives_of_rows_in_any_order(tmp_path):
    assert "score: ok" in _run(tmp_path, "logprob.hip", "score_check.cpp")


def test_order_of_tokens(tmp_path):
    shared = ("extern __shared__ uint32_t places[];", "static uint32_t places[ORDER_WAVES << 9];")
    assert "order: ok" in _run(tmp_path, "embed.hip", "order_check.cpp", [shared])
