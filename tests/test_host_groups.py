"""The validation and planning of the grouped and MXFP4 entry points (pure host C++) under g++'s address and
undefined-behaviour sanitizers, driven by tests/csrc/host_checks_groups.cpp."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_code_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    csrc = os.path.join(ROOT, "fp8_blockwise_quantized_amd", "csrc")
    exe = str(tmp_path / "host_checks_groups")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", csrc,
           os.path.join(ROOT, "tests", "csrc", "host_checks_groups.cpp"), os.path.join(csrc, "validate.cpp"),
           os.path.join(csrc, "plan.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
